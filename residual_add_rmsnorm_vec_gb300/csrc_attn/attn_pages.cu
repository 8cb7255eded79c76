// A serving step's plan from the requests' lengths: pages returned and taken,
// block table, positions, slots.
//
// What bounds it: latency.  A step of 1024 sequences reads 12 KB and writes 30;
// the chain is lengths -> three block scans (rows, returned pages, taken pages) and a
// maximum, eight barriers -> free list -> stores.  8 sequences x 1 token 4.8 us, 1024 x 1 7.0
// (9.6 with 5 % finished), 64 x 2000 tokens 7.5 (9.0).  So one launch, and
// no exchange between blocks: with up to kPagesOnce sequences every block scans
// all of them for itself into shared memory (12 bytes a sequence from L2) and
// then plans its own rows.  Larger batches scan once, in a first launch of one
// block, into the workspace; that block then bounds them (2048 x 1 8.2 us, 2049 x 1 11.5,
// 4096 x 1 14.8, 16384 x 1 63).
//
// Nothing that a block writes is read by another one: the free list is read
// below n_free and written from there on, the table's new entries are found from
// the free list again by every row that needs them, and the count goes out to a
// word of its own.  The same inputs thus give the same results however often the
// call is made.
#include "attn_common.cuh"

namespace rmsattn {

namespace {

// What the scan leaves for a sequence.
//   cu     its first row, at most T
//   base   pages taken by earlier sequences; -1: left out, finished or empty
//   back   pages returned by earlier sequences, at most n_pages
struct Scan {
    int32_t *cu, *base, *back;  // cu and back: one more, behind the last
    int32_t top;                // free pages once all are returned
    int32_t left;               // free pages in the end
    int32_t count;              // free pages before
};

// Pages of x < 2^32 tokens.
__device__ __forceinline__ uint32_t pages_of(uint32_t x, uint32_t page) {
    const uint32_t q = x / page;
    return q + (q * page != x);
}

// What a sequence holds, gets and keeps when it is finished.
struct Word {
    int32_t len, more, kept;
    __device__ __forceinline__ void of(const PagesArgs& a, int64_t s) {
        len = a.lengths[s];
        more = a.more[s];
        kept = a.shared ? a.shared[s] : 0;
        if (kept < 0) kept = 0;
    }
};
// A sequence as the scan sees it.
struct Seq {
    int32_t len;
    uint32_t more, has, need;
    int64_t back;
    bool live, done;
    __device__ __forceinline__ void of(const PagesArgs& a, const Word& w) {
        len = w.len < 0 ? 0 : w.len;
        live = w.len >= 0;
        done = live && w.more < 0;
        more = live && w.more > 0 ? (uint32_t)w.more : 0u;
        has = pages_of((uint32_t)len, (uint32_t)a.page);
        need = pages_of((uint32_t)len + more, (uint32_t)a.page);
        back = 0;
        if (done) {
            const int64_t own = has < a.width ? has : a.width;
            back = own > w.kept ? own - w.kept : 0;
        }
    }
    __device__ __forceinline__ bool fits(const PagesArgs& a, int64_t begin) const {
        return live && !done && need <= a.width && begin + more <= a.T && (int64_t)len + more <= INT32_MAX;
    }
    __device__ __forceinline__ uint32_t take() const { return need - has; }
};

// Exclusive sum over the block of one value a thread, and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t* total) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();  // an earlier scan's sums have been read
    if (lane == 31) sums[wp] = inc;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < wp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + inc - v;
}

__device__ __forceinline__ int32_t clamp_to(int64_t v, int64_t most) {
    return (int32_t)(v < most ? v : most);
}

// All sequences, a run of them to each thread; of a run's first kHeld the words stay in
// registers.
__device__ __forceinline__ void scan(const PagesArgs& a, Scan* sc) {
    constexpr int kHeld = 4;
    __shared__ int64_t sums[32];
    __shared__ int32_t most[32];
    const int64_t per = (a.B + blockDim.x - 1) / blockDim.x, s0 = threadIdx.x * per;
    const int64_t s1 = s0 + per < a.B ? s0 + per : a.B;
    int64_t count = *a.n_free;
    Word held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        held[i].len = -1;
        if (s0 + i < s1) held[i].of(a, s0 + i);
    }
    count = count < 0 ? 0 : (count < a.n_pages ? count : a.n_pages);
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (s0 + i < s1) f(s0 + i, held[i]);
        for (int64_t s = s0 + kHeld; s < s1; ++s) {
            Word w;
            w.of(a, s);
            f(s, w);
        }
    };
    int64_t rows = 0, back = 0;
    each([&](int64_t, const Word& w) {
        Seq q;
        q.of(a, w);
        rows += q.more;
        back += q.back;
    });
    int64_t all_rows, all_back, all_taken;
    int64_t begin = block_scan(rows, sums, &all_rows), from = block_scan(back, sums, &all_back);
    const int64_t top = count + all_back < a.n_pages ? count + all_back : a.n_pages;
    if (count + all_back > a.n_pages && threadIdx.x == 0) atomicOr(a.status, kBadPage);
    int64_t taken = 0, b = begin;
    each([&](int64_t, const Word& w) {
        Seq q;
        q.of(a, w);
        if (q.fits(a, b)) taken += q.take();
        b += q.more;
    });
    int64_t at = block_scan(taken, sums, &all_taken), out = 0;
    each([&](int64_t s, const Word& w) {
        Seq q;
        q.of(a, w);
        sc->cu[s] = clamp_to(begin, a.T);
        sc->back[s] = clamp_to(from, a.n_pages);
        int32_t base = -1;
        if (q.fits(a, begin)) {
            const uint32_t n = q.take();
            if (n == 0 || at + n <= top) {
                base = clamp_to(at, INT32_MAX);
                if (n > 0) out = at + n;
            }
            at += n;
        }
        sc->base[s] = base;
        begin += q.more;
        from += q.back;
    });
    if (s1 == a.B && s0 < s1) {
        sc->cu[a.B] = clamp_to(begin, a.T);
        sc->back[a.B] = clamp_to(from, a.n_pages);
    }
    if (a.B == 0 && threadIdx.x == 0) sc->cu[0] = sc->back[0] = 0;
    // the last page that went out
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int32_t m = __reduce_max_sync(0xFFFFFFFFu, (int32_t)out);
    if (lane == 0) most[wp] = m;
    __syncthreads();
    int32_t last = 0;
    for (int w = 0; w < nw; ++w) last = most[w] > last ? most[w] : last;
    sc->count = (int32_t)count;
    sc->top = (int32_t)top;
    sc->left = (int32_t)(top - last);
}

// The last of v[0 .. n - 1] (non-decreasing, v[0] <= x) that is at most x.
__device__ __forceinline__ int64_t last_at_most(const int32_t* v, int64_t n, int32_t x) {
    int64_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t kept(const PagesArgs& a, int64_t s) {
    const int32_t k = a.shared ? a.shared[s] : 0;
    return k < 0 ? 0 : k;
}

// Entry i of the free pages with the returned ones behind them.
__device__ __forceinline__ int32_t page_at(const PagesArgs& a, const Scan& sc, int32_t i) {
    if (i < sc.count) return a.free_pages[i];
    const int32_t f = i - sc.count;
    const int64_t s = last_at_most(sc.back, a.B, f);
    return a.table[s * a.table_stride + kept(a, s) + f - sc.back[s]];
}

// Rows U t to U t + U - 1 of the batch for thread t.
template <int U>
__device__ __forceinline__ void each_row(const PagesArgs& a, const Scan& sc, int64_t me, int64_t threads) {
    const int32_t all = sc.cu[a.B];
    for (int64_t t0 = me * U; t0 < a.T; t0 += threads * U) {
        int32_t pos[U], row[U];
        int64_t slot[U];
        int64_t s = t0 < all ? last_at_most(sc.cu, a.B, (int32_t)t0) : 0;
        int64_t at = -1;  // the sequence that len and has are of
        int32_t len = 0, base = -1;
        uint32_t has = 0;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int32_t t = (int32_t)(t0 + k);
            pos[k] = 0;
            row[k] = -1;
            slot[k] = -1;
            if (t >= all) continue;
            while (sc.cu[s + 1] <= t) ++s;
            if (s != at) {
                at = s;
                len = a.lengths[s];
                has = pages_of((uint32_t)len, (uint32_t)a.page);
                base = sc.base[s];
            }
            const uint32_t p = (uint32_t)len + (uint32_t)(t - sc.cu[s]);
            pos[k] = (int32_t)p;
            row[k] = (int32_t)s;
            if (base < 0) continue;
            const uint32_t j = p / (uint32_t)a.page;
            int32_t* entry = a.table + s * a.table_stride + j;
            int32_t page;
            if (j < has) {
                page = *entry;
            } else {
                page = page_at(a, sc, sc.top - 1 - (base + (int32_t)(j - has)));
                if (p == j * a.page) *entry = page;  // the page's first row brings it in
            }
            if ((uint32_t)page < (uint32_t)a.n_pages) slot[k] = (int64_t)page * a.page + (p - j * a.page);
            else atomicOr(a.status, kBadPage);
        }
        if (U == 4 && t0 + 4 <= a.T) {
            *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[U / 4], pos[U / 2], pos[U - 1]);
            *reinterpret_cast<int4*>(a.rows + t0) = make_int4(row[0], row[U / 4], row[U / 2], row[U - 1]);
            *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[U / 4]);
            *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[U / 2], slot[U - 1]);
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (t0 + k >= a.T) break;
                a.positions[t0 + k] = pos[k];
                a.rows[t0 + k] = row[k];
                a.slots[t0 + k] = slot[k];
            }
        }
    }
}

__device__ __forceinline__ void plan_rows(const PagesArgs& a, const Scan& sc) {
    const int64_t threads = (int64_t)gridDim.x * blockDim.x, me = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    // sequences
    for (int64_t s = me; s < a.B; s += threads) {
        const int32_t len = a.lengths[s], more = a.more[s];
        const bool ok = sc.base[s] >= 0;  // (then len is not negative, nor is more)
        a.cu[s] = sc.cu[s];
        a.before[s] = ok ? len : -1;
        a.after[s] = ok ? len + more : (len >= 0 && more < 0 ? 0 : len);
    }
    if (me == 0) {
        a.cu[a.B] = sc.cu[a.B];
        *a.n_free_out = sc.left;
    }
    // returned pages, a warp to a sequence
    for (int64_t s = me >> 5; s < a.B; s += threads >> 5) {
        const int32_t f0 = sc.back[s], f1 = sc.back[s + 1];
        if (f0 == f1) continue;
        const int32_t* row = a.table + s * a.table_stride + kept(a, s);
#pragma unroll 4
        for (int32_t f = f0 + (threadIdx.x & 31); f < f1; f += 32) {
            const int32_t p = row[f - f0];
            if ((uint32_t)p >= (uint32_t)a.n_pages) atomicOr(a.status, kBadPage);
            if (sc.count + f < sc.left) a.free_pages[sc.count + f] = p;
        }
    }
    // rows: four to a thread (and whole vectors to write) where there are two or more, else
    // one, whose chain of loads nothing lengthens (64 x 2000 tokens take 0.89 of the time with
    // four, 1024 x 1 1.23 of it)
    if (a.T >= 2 * threads) each_row<4>(a, sc, me, threads);
    else each_row<1>(a, sc, me, threads);
}

__global__ void __launch_bounds__(512) pages_kernel(const PagesArgs a) {
    extern __shared__ int32_t seqs[];
    rmsn::pdl_wait(a.pdl);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Scan sc;
    sc.cu = seqs;
    sc.back = seqs + a.B + 1;
    sc.base = seqs + 2 * (a.B + 1);
    scan(a, &sc);
    __syncthreads();
    plan_rows(a, sc);
}

// The workspace: three counts, then cu, back and base.
__global__ void __launch_bounds__(1024) pages_scan_kernel(const PagesArgs a) {
    rmsn::pdl_wait(a.pdl);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Scan sc;
    sc.cu = a.ws + 4;
    sc.back = sc.cu + a.B + 1;
    sc.base = sc.back + a.B + 1;
    scan(a, &sc);
    if (threadIdx.x == 0) {
        a.ws[0] = sc.top;
        a.ws[1] = sc.left;
        a.ws[2] = sc.count;
    }
}

__global__ void __launch_bounds__(512) pages_rows_kernel(const PagesArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Scan sc;
    sc.cu = a.ws + 4;
    sc.back = sc.cu + a.B + 1;
    sc.base = sc.back + a.B + 1;
    sc.top = a.ws[0];
    sc.left = a.ws[1];
    sc.count = a.ws[2];
    plan_rows(a, sc);
}

}  // namespace

const void* pages_kernel_of(int which) {
    return which == 0 ? (const void*)&pages_kernel
                      : (which == 1 ? (const void*)&pages_scan_kernel : (const void*)&pages_rows_kernel);
}

}  // namespace rmsattn
