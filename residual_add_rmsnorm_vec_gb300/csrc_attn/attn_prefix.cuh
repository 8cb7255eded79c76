// Attention of a group's queries over the tokens that the group shares: the parts
// that attn_attend.cuh's kernels add to each sequence's own tokens.
//
//   s_j = scale q . k_j,  l = sum exp(s_j - m),  O = sum exp(s_j - m) v_j
//
// A row is one column of the group (sequence x query token x head of a key head).
// All of a group's rows meet the same keys and values, so the products are matrix
// products: 4 D flops for each pair of a row and a token against 2 D + 1/2 bytes a
// token.  From about 150 rows on the tensor cores bound it, below that DRAM.
//
// A block holds R tiles of 128 rows (R = 2 where a group has more than 128 rows)
// and walks over its share of the line of all steps, TOK tokens of an item (group x
// key head x R tiles) each.  Its warps have fixed parts:
//
//   softmax  four warps to a row tile, a thread to a row: scores from TMEM, weights
//            back into TMEM as the second product's A operand, in fp16
//   K, V     four warps: codes from the pages (16-byte loads, a tile's on their way in
//            registers while the stages are full), widened to fp16 into the swizzled
//            stages of the B operands
//   MMA      one warp, one of its lanes issues: for each row tile O += P V of the step
//            before, then S = Q K^T of this one; the other row tile's softmax runs
//            meanwhile
//
// * Widening 16-bit copies into shared memory pays here, other than in attn_attend.cuh:
//   256 rows use each copy.
// * A value's scale is 2^e times a significand in [1, 2).  The significand multiplies
//   the weight before that is rounded to fp16 (the one rounding of the weight: half a
//   step, 2^-11), 2^e the codes: code * 2^(7 + e - E) is exact in fp16 for e in
//   [E - 22, E].  E is the block's reference; a block of tokens outside its window makes
//   a step of its own, for which what was summed so far is added to the part in memory
//   and E set anew.  Scales that lie 2^22 apart are rare, so that path is small.
// * A row's reference m follows its maximum only when that has grown by more than
//   2^kSlack; then the row's sum is multiplied in TMEM by the softmax warp itself: the
//   commit that announced the scores covers the product before them.  Weights are
//   lifted by kLift: a lifted weight times a significand stays below 2^15, and fp16's
//   subnormals end 2^-34 below the reference.
// * Parts go to the workspace in the order of the line: nothing depends on timing.
// * Every wait gives up after a second: the block then stops, waits for its products
//   in flight, gives TMEM back, and bit 0 of the status word is set.
#pragma once

#include "attn_common.cuh"

namespace rmsattn {
namespace prefix {

using rmsn::F2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.402823466e38f;  // the reference before any token is seen
constexpr float kSlack = 5.f;
constexpr int kLiftLog = 9;
constexpr float kLift = 512.f;
constexpr float kWide = 4194304.f;  // 2^22: up to it, a product's rounding error is 2^-3 at most
constexpr long long kWaitCycles = 2000000000LL;

// flags of a step
constexpr uint32_t kFirst = 1u, kLast = 2u, kFlush = 4u, kEnd = 8u, kTwo = 16u;

template <int D_, int R_>
struct Shape {
    static constexpr int D = D_, R = R_;
    static constexpr int TOK = D == 256 ? 64 : 128;
    static constexpr int BLK = TOK / kBlock;
    static constexpr int PARTS = D / 64;              // 64-dim parts of 128-byte lines
    static constexpr int S = D == 64 ? 3 : 2;         // stages of K and of V
    static constexpr int M = 4;                       // slots of the steps' words, >= S + 2
    static constexpr int kTile = TOK * D * 2;
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kSmem = R * kQ + 2 * S * kTile + 1024;
    static constexpr int kThreads = (4 * R + 5) * 32;
    static constexpr int kCols = 512;                 // of TMEM: S at 128 x, O behind
    static constexpr int kO = 256;
    static constexpr int ITERS = TOK / 8 * PARTS / 4; // 16-byte loads of a thread and tile
};

struct Step {
    float ks[8], vm[8];
    uint32_t mask, flags;
    int32_t e, pad;
};

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float exp2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Shared-memory operand: rows of 128 bytes, 128-byte swizzle, eight rows to 1024
// bytes; `lead`: bytes between 64-element parts of an operand whose rows are the
// product's inner dimension.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           uint64_t(1) << 46 | uint64_t(2) << 61;
}
// fp16 operands, fp32 sums, 128 rows, n columns; `inner`: B's rows are the inner dimension.
__host__ __device__ constexpr uint32_t product(int n, bool inner) {
    return 1u << 4 | (inner ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// 32 columns of the warp's 32 rows, waited for.
__device__ __forceinline__ void tmem_load(float (&v)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
        "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]),
        "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]),
        "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- the block

struct Bars {
    uint64_t k_full[4], k_free[4], v_full[4], v_free[4], step[4], s_full[2], p_full[2], q_full[2], o_done[2], last;
    uint32_t tmem, stop;
};

// All of a warp's lanes wait together, for a second at most; false: the block stops.
__device__ __forceinline__ bool wait(const uint64_t* bar, uint32_t parity, uint32_t* stop) {
    const uint32_t b = smem_of(bar);
    bool ok = rmsn::mbar_try_wait(b, parity & 1);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
        const long long t0 = clock64();
        while (!__all_sync(0xFFFFFFFFu, ok)) {
            if (!ok) ok = rmsn::mbar_try_wait(b, parity & 1);
            const bool out = *reinterpret_cast<volatile uint32_t*>(stop) != 0 || clock64() - t0 > kWaitCycles;
            if (__any_sync(0xFFFFFFFFu, out && !ok)) {
                *reinterpret_cast<volatile uint32_t*>(stop) = 1;
                return false;
            }
        }
    }
    return true;
}

// A block's piece of an item: `steps` of its steps from `step0` on.
struct Piece {
    int hk, tile, step0, steps, item;  // item: counted over all groups
    PrefixGroup g;
};

// The pieces of a share, in the line's order.
struct Walk {
    int at, stop, g;
    __device__ __forceinline__ void begin(const PrefixArgs& a) {
        const PrefixLine line = *a.line;
        const int64_t from = (int64_t)blockIdx.x * line.chunk, to = from + line.chunk;
        at = (int)(from < line.total ? from : line.total);
        stop = (int)(to < line.total ? to : line.total);
        g = 0;
        if (at < stop) {  // the last group that begins at `at` or before; groups without steps begin where the next does
            int hi = a.n_groups;
            while (hi - g > 1) {
                const int mid = (g + hi) >> 1;
                if (a.groups[mid].first <= at) g = mid;
                else hi = mid;
            }
        }
    }
    __device__ __forceinline__ bool next(const PrefixArgs& a, Piece* p) {
        if (at >= stop) return false;
        for (;;) {
            p->g = a.groups[g];
            if (p->g.ns > 0 && at < p->g.first + p->g.ns * p->g.tiles * a.c.H) break;
            ++g;
        }
        const int item = (at - p->g.first) / p->g.ns;
        p->step0 = (at - p->g.first) - item * p->g.ns;
        const int left = p->g.ns - p->step0;
        p->steps = stop - at < left ? stop - at : left;
        p->hk = item / p->g.tiles;
        p->tile = item - p->hk * p->g.tiles;
        p->item = p->g.item0 + item;
        at += p->steps;
        return true;
    }
};

// A tile of TOK tokens as a producer warp sees it: lane b (< BLK) has block b.
struct Tile {
    bool on, first, last;  // on: there is one; first / last of its piece
    bool two;              // the second row tile has rows
    int hk, j;             // its first token
    int shared;
    const int32_t* row;
};

template <class C>
struct Tiles {
    Walk walk;
    Piece p;
    int step;
    bool more;
    __device__ __forceinline__ void begin(const PrefixArgs& a) {
        walk.begin(a);
        more = walk.next(a, &p);
        step = 0;
    }
    __device__ __forceinline__ void next(const PrefixArgs& a, Tile* t) {
        t->on = more;
        if (!more) return;
        t->first = step == 0;
        t->last = step == p.steps - 1;
        t->hk = p.hk;
        t->j = (p.step0 + step) * C::TOK;
        t->shared = p.g.shared;
        t->row = a.table + p.g.seq * a.table_stride;
        t->two = C::R == 2 && ((p.g.s1 - p.g.s0) * a.n * a.group - p.tile * (128 * C::R)) > 128;
        if (++step == p.steps) {
            more = walk.next(a, &p);
            step = 0;
        }
    }
};

// Page of the lane's block, or -1 (no such block, or no such page).
template <class C>
__device__ __forceinline__ int32_t page_entry(const PrefixArgs& a, const Tile& t, int lane, int* at) {
    const int j = t.j + lane * kBlock;
    *at = 0;
    if (!t.on || lane >= C::BLK || j >= t.shared) return -1;
    const int slot = (int)(((uint64_t)(uint32_t)(j >> 4) * a.page_rcp) >> 37);
    *at = (j - slot * a.c.page) >> 4;
    const int32_t page = t.row[slot];
    if ((uint32_t)page >= (uint32_t)a.c.n_pages) {
        atomicOr(a.status, kBadPage);
        return -1;
    }
    return page;
}

// The four warps that fill the stages of K and V and write the steps' words.
template <class C>
__device__ __forceinline__ void produce(const PrefixArgs& a, unsigned char* stages, Bars* bars, Step* steps, int wp) {
    constexpr int D = C::D;
    const int lane = threadIdx.x & 31;
    Tiles<C> tiles;
    tiles.begin(a);
    Tile t;
    tiles.next(a, &t);
    int at;
    int32_t page = page_entry<C>(a, t, lane, &at);
    // this lane's 16 bytes of eight tokens' 64 dims: a quarter warp's stores (two
    // tokens whose numbers differ in bit 0, four chunks each) meet all banks
    const int r8 = (lane >> 3) * 2 + ((lane >> 2) & 1), c4 = lane & 3;
    const int mine = r8 * D + c4 * 16;
    uint4 kv[2][C::ITERS];
    int n = 0;  // steps so far
    int E = 0;  // the piece's reference
    while (t.on) {
        // the tile's scales and codes
        const int64_t tile = (int64_t)t.hk * (a.c.page >> 4) + at;
        const bool have = page >= 0;
        float ks = 0.f, vs = 0.f;
        if (have) {
            const int64_t i = (int64_t)page * a.c.scale_stride + tile;
            ks = a.c.ks[i];
            vs = a.c.vs[i];
        }
        const int64_t off = have ? (int64_t)page * a.c.page_stride + tile * (kBlock * D) : -1;
        uint32_t rem = __ballot_sync(0xFFFFFFFFu, have);
#pragma unroll
        for (int i = 0; i < C::ITERS; ++i) {
            const int u = i * 4 + wp, tg = u / C::PARTS, h = u % C::PARTS;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, tg >> 1);
            kv[0][i] = kv[1][i] = make_uint4(0, 0, 0, 0);
            if (o >= 0) {
                const int64_t e = o + ((tg & 1) * 8 * D + h * 64 + mine);
                kv[0][i] = rmsn::ld_stream16(a.c.k + e);
                kv[1][i] = rmsn::ld_stream16(a.c.v + e);
            }
        }
        bool begin = t.first;
        const bool last = t.last, two = t.two;
        tiles.next(a, &t);
        page = page_entry<C>(a, t, lane, &at);
        // the lane's value scale: 2^e vm, vm in [1, 2); 0 fits any reference
        uint32_t bits = __float_as_uint(vs) & 0x7FFFFFFFu;
        int down = 0;
        if (bits != 0 && bits < 0x00800000u) {  // below fp32's normal range
            bits = __float_as_uint(__uint_as_float(bits) * 16777216.f);
            down = 24;
        }
        const bool zero = bits == 0;
        const int e = (int)(bits >> 23) - 127 - down;
        const float vm = zero ? 1.f : __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
        do {
            uint32_t flags = (begin ? kFirst : 0u) | (two ? kTwo : 0u);
            auto fitting = [&]() { return __ballot_sync(0xFFFFFFFFu, zero || (e <= E && e >= E - 22)) & rem; };
            uint32_t mask = fitting();
            if (begin || (rem != 0 && mask == 0)) {
                const int top = __reduce_max_sync(0xFFFFFFFFu, !zero && (rem >> lane & 1) ? e : -1000);
                if (!begin) flags |= kFlush;
                E = top == -1000 ? 0 : top + 3;
                mask = fitting();
            }
            rem &= ~mask;
            if (rem == 0 && last) flags |= kLast;
            begin = false;
            const int st = n % C::S;
            const uint32_t turn = (uint32_t)(n / C::S + 1);
            if (!wait(&bars->k_free[st], turn, &bars->stop)) return;
            if (wp == 0) {
                Step* w = steps + n % C::M;
                if (lane < C::BLK) {
                    w->ks[lane] = ks;
                    w->vm[lane] = vm * kLift;
                }
                if (lane == 0) {
                    w->mask = mask;
                    w->flags = flags;
                    w->e = E;
                }
                __syncwarp();
                if (lane == 0) arrive(smem_of(&bars->step[n % C::M]));
            }
            // 2^(7 + e - E) as packed fp16
            const int k7 = 7 + e - E;
            uint32_t f = zero ? 0u : (k7 >= -14 ? (uint32_t)(k7 + 15) << 10 : 0x200u);
            f |= f << 16;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (v && !wait(&bars->v_free[st], turn, &bars->stop)) return;
                const uint32_t dst = smem_of(stages) + (v * C::S + st) * C::kTile;
#pragma unroll
                for (int i = 0; i < C::ITERS; ++i) {
                    const int u = i * 4 + wp, tg = u / C::PARTS, h = u % C::PARTS;
                    const uint32_t w[4] = {kv[v][i].x, kv[v][i].y, kv[v][i].z, kv[v][i].w};
                    uint32_t y[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        y[2 * k] = e4m3x2_to_f16x2(w[k]);
                        y[2 * k + 1] = e4m3x2_to_f16x2(w[k] >> 16);
                    }
                    if (v) {
                        const uint32_t fb = __shfl_sync(0xFFFFFFFFu, f, tg >> 1);
                        const bool on = mask >> (tg >> 1) & 1;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y[k]) : "r"(fb));
                            if (!on) y[k] = 0u;  // (a NaN code times 0 is not)
                        }
                    }
                    const int r = tg * 8 + r8;
                    const uint32_t line = dst + h * (C::TOK * 128) + r * 128;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                         line + (((2 * c4 + k) ^ (r & 7)) << 4)),
                                     "r"(y[4 * k]), "r"(y[4 * k + 1]), "r"(y[4 * k + 2]), "r"(y[4 * k + 3])
                                     : "memory");
                }
                fence_async();
                __syncwarp();
                if (lane == 0) arrive(smem_of(v ? &bars->v_full[st] : &bars->k_full[st]));
            }
            ++n;
        } while (rem != 0);
    }
    // one more step's word: there are none left
    const int st = n % C::S;
    if (!wait(&bars->k_free[st], (uint32_t)(n / C::S + 1), &bars->stop)) return;
    if (wp == 0 && lane == 0) {
        steps[n % C::M].flags = kEnd;
        arrive(smem_of(&bars->step[n % C::M]));
    }
    __syncwarp();
    if (lane == 0) arrive(smem_of(&bars->k_full[st]));
}

// The warp that issues the products.
template <class C>
__device__ __forceinline__ void multiply(unsigned char* smem, Bars* bars, const Step* steps) {
    constexpr uint32_t kS = product(C::TOK, false), kP = product(C::D, true);
    const int lane = threadIdx.x & 31;
    const uint32_t q_at = smem_of(smem), k_at = q_at + C::R * C::kQ, v_at = k_at + C::S * C::kTile;
    const uint32_t tmem = bars->tmem;
    uint32_t p_turn[2] = {0, 0}, q_turn[2] = {0, 0};
    uint32_t was = 0;  // flags of the step before
    for (int n = 0;; ++n) {
        const int st = n % C::S, pst = (n - 1) % C::S;
        if (!wait(&bars->k_full[st], (uint32_t)(n / C::S), &bars->stop)) break;
        const uint32_t flags = steps[n % C::M].flags;
        if (n > 0 && !wait(&bars->v_full[pst], (uint32_t)((n - 1) / C::S), &bars->stop)) break;
        bool ok = true;
#pragma unroll
        for (int x = 0; x < C::R; ++x) {
            if (n > 0) {
                if (!(ok = wait(&bars->p_full[x], p_turn[x]++, &bars->stop))) break;
                tc_after();
                if (lane == 0) {
                    if (x == 0 || (was & kTwo)) {
                        const uint32_t o = tmem + C::kO + x * C::D, p = tmem + x * 128;
                        const bool fresh = was & (kFirst | kFlush);
#pragma unroll
                        for (int k = 0; k < C::TOK / 16; ++k)
                            mma_ts(o, p + k * 8, operand(v_at + pst * C::kTile + k * 2048, C::TOK * 128), kP,
                                   !(fresh && k == 0));
                        if (was & kLast) commit(smem_of(&bars->o_done[x]));
                    }
                    if (x == C::R - 1) commit(smem_of(&bars->v_free[pst]));
                }
                __syncwarp();
            }
            if (!(flags & kEnd)) {  // (a row tile without rows keeps step with the other)
                const bool on = x == 0 || (flags & kTwo);
                if (on && (flags & kFirst) && !(ok = wait(&bars->q_full[x], q_turn[x]++, &bars->stop))) break;
                tc_after();
                if (lane == 0) {
                    if (on) {
#pragma unroll
                        for (int k = 0; k < C::D / 16; ++k)
                            mma_ss(tmem + x * 128,
                                   operand(q_at + x * C::kQ + (k / 4) * (128 * 128) + (k % 4) * 32, 16),
                                   operand(k_at + st * C::kTile + (k / 4) * (C::TOK * 128) + (k % 4) * 32, 16), kS,
                                   k > 0);
                    }
                    commit(smem_of(&bars->s_full[x]));
                }
                __syncwarp();
            }
        }
        if (!ok || (flags & kEnd)) break;
        if (lane == 0) commit(smem_of(&bars->k_free[st]));
        __syncwarp();
        was = flags;
    }
    // nothing is in flight when the block leaves
    if (lane == 0) commit(smem_of(&bars->last));
    __syncwarp();
    const long long t0 = clock64();
    while (!rmsn::mbar_try_wait(smem_of(&bars->last), 0) && clock64() - t0 < kWaitCycles) {
    }
}

// The four warps of row tile x.
template <class T, class C>
__device__ __forceinline__ void soften(const PrefixArgs& a, unsigned char* smem, Bars* bars, const Step* steps, int x) {
    constexpr int D = C::D, ROWS = 128 * C::R;
    const int wp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, r = wp * 32 + lane;
    const uint32_t lanes = (uint32_t)(wp * 32) << 16;
    const uint32_t s_at = bars->tmem + lanes + x * 128, o_at = bars->tmem + lanes + C::kO + x * D;
    unsigned char* q_rows = smem + x * C::kQ;
    Walk walk;
    walk.begin(a);
    Piece p;
    uint32_t s_turn = 0, o_turn = 0;
    int n = 0;  // steps of the block so far
    float q_scale = 0.f, q_next = 0.f;
    int valid = 0, valid_next = 0;  // rows of this tile
    // the piece's queries, scaled to fp16 by a power of two as in attn_attend.cuh
    auto load_q = [&]() {
        const int cols = (p.g.s1 - p.g.s0) * a.n * a.group - p.tile * ROWS - x * 128;
        valid_next = cols < 0 ? 0 : cols;
        if (valid_next == 0) return;  // (x == 1 alone: the products leave it out)
        q_next = 0.f;
        if (r >= valid_next) {  // rows of nothing: scores of 0
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(q_rows + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(0, 0, 0, 0);
        } else {
            const int cc = p.tile * ROWS + x * 128 + r, token = cc / a.group;
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + ((int64_t)p.g.s0 * a.n + token) * a.q_stride +
                                  (int64_t)(p.hk * a.group + cc - token * a.group) * D;
            constexpr int H = 64;  // dims held at once
            uint4 v[H / 8];
            float m = 0.f;
#pragma unroll 1
            for (int d0 = D - H; d0 >= 0; d0 -= H) {
#pragma unroll
                for (int i = 0; i < H / 8; ++i) v[i] = *reinterpret_cast<const uint4*>(src + d0 + i * 8);
#pragma unroll
                for (int i = 0; i < H / 8; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // (a maximum leaves NaN out; its products find it)
                        m = rmsn::absmax3(m, rmsn::lo2<T>(w[k]), rmsn::hi2<T>(w[k]));
                    }
                }
            }
            int e = (int)(__float_as_uint(m) >> 23) - 127 - 7;
            e = e < -126 ? -126 : (e > 126 ? 126 : e);
            const float down = m > 3.402823466e38f ? __uint_as_float(0x7FFFFFFFu)
                                                   : copysignf(pow2(-e), a.scale);
            q_next = pow2(e) * (fabsf(a.scale) * kLog2e);
#pragma unroll 1
            for (int d0 = 0; d0 < D; d0 += H) {  // (the first are still there)
                if (d0 > 0) {
#pragma unroll
                    for (int i = 0; i < H / 8; ++i) v[i] = *reinterpret_cast<const uint4*>(src + d0 + i * 8);
                }
#pragma unroll
                for (int i = 0; i < H / 8; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y[k] = rmsn::pack_f16x2(rmsn::lo2<T>(w[k]) * down, rmsn::hi2<T>(w[k]) * down);
                    const int c = d0 / 8 + i;
                    *reinterpret_cast<uint4*>(q_rows + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) arrive(smem_of(&bars->q_full[x]));
    };
    bool more = walk.next(a, &p);
    if (more) load_q();
    while (more) {
        const Piece now = p;
        q_scale = q_next;
        valid = valid_next;
        const bool busy = wp * 32 < valid;  // the warp has rows
        float* part = a.parts + ((int64_t)blockIdx.x + now.item) * (ROWS * (int64_t)(D + 2)) + (x * 128 + r) * 8;
        float ref = kNone, l = 0.f;
        float part_ref = 0.f;
        bool has_part = false;
        int E = 0;
        // what O holds goes to the part, in units of the reference
        auto drain = [&]() {
            const int up = E - 7 - kLiftLog, half = up >> 1;  // 2^up in two steps: it may lie outside fp32's range
            const float f0 = pow2(half), f1 = pow2(up - half);
            const float keep = has_part ? exp2a(part_ref - ref) : 0.f;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                float o[32];
                tmem_load(o, o_at + d);
                if (r < valid) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float4* y = reinterpret_cast<float4*>(part + (d / 8 + i / 8) * (ROWS * 8) + (i & 4));
                        float4 v = make_float4(o[i] * f0 * f1, o[i + 1] * f0 * f1, o[i + 2] * f0 * f1, o[i + 3] * f0 * f1);
                        if (has_part) {
                            const float4 w = *y;
                            v = make_float4(v.x + w.x * keep, v.y + w.y * keep, v.z + w.z * keep, v.w + w.w * keep);
                        }
                        *y = v;
                    }
                }
            }
            has_part = true;
            part_ref = ref;
        };
        uint32_t flags = 0;
        if (valid > 0 || x == 0) {
            do {
                const Step* w = steps + n % C::M;
                if (!wait(&bars->step[n % C::M], (uint32_t)(n / C::M), &bars->stop)) return;
                if (!wait(&bars->s_full[x], s_turn++, &bars->stop)) return;
                tc_after();
                flags = w->flags;
                if (busy) {
                    const uint32_t mask = w->mask;
                    if (flags & kFlush) drain();
                    E = w->e;
                    // the row's maximum
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < C::TOK; c += 32) {
                        float s[32];
                        tmem_load(s, s_at + c);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(mask >> (c / 16 + h) & 1)) continue;
                            const float kc = w->ks[c / 16 + h] * q_scale;
                            float m = -INFINITY;  // of the scores before the factor, which is not negative
#pragma unroll
                            for (int i = 0; i < 16; i += 2) m = max3(m, s[16 * h + i], s[16 * h + i + 1]);
                            top = fmaxf(top, __fmul_rn(m, kc));
                        }
                    }
                    if (__any_sync(0xFFFFFFFFu, top > ref + kSlack)) {
                        const float to = fmaxf(ref, top), keep = exp2a(ref - to);
                        ref = to;
                        l *= keep;
                        if (!(flags & (kFirst | kFlush))) {
#pragma unroll 1
                            for (int d = 0; d < D; d += 32) {
                                float o[32];
                                tmem_load(o, o_at + d);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= keep;
                                tmem_store32(o_at + d, o);
                            }
                            tmem_stored();
                        }
                    }
                    // the weights
                    const bool wide = __any_sync(0xFFFFFFFFu, fabsf(ref) > kWide && ref != kNone);
                    F2 sum = rmsn::f2(0.f, 0.f);
                    const F2 less = rmsn::f2(-ref, -ref);
#pragma unroll 1
                    for (int c = 0; c < C::TOK; c += 32) {
                        float s[32];
                        uint32_t y[16];
                        tmem_load(s, s_at + c);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(mask >> (c / 16 + h) & 1)) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[8 * h + i] = 0u;
                                continue;
                            }
                            const float kc = w->ks[c / 16 + h] * q_scale, vm = w->vm[c / 16 + h];
                            const F2 kc2 = rmsn::f2(kc, kc), vm2 = rmsn::f2(vm, vm);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float lo = s[16 * h + 2 * i], hi = s[16 * h + 2 * i + 1];
                                if (wide) {
                                    lo = __fsub_rn(__fmul_rn(lo, kc), ref);
                                    hi = __fsub_rn(__fmul_rn(hi, kc), ref);
                                } else {
                                    rmsn::f2split(rmsn::fma2(rmsn::f2(lo, hi), kc2, less), lo, hi);
                                }
                                const F2 pp = rmsn::f2(exp2a(lo), exp2a(hi));
                                sum = rmsn::add2(sum, pp);
                                rmsn::f2split(rmsn::mul2(pp, vm2), lo, hi);
                                y[8 * h + i] = rmsn::pack_f16x2(lo, hi);
                            }
                        }
                        tmem_store16(s_at + c / 2, y);
                    }
                    float lo, hi;
                    rmsn::f2split(sum, lo, hi);
                    l += lo + hi;
                    tmem_stored();
                }
                tc_before();
                __syncwarp();
                if (lane == 0) arrive(smem_of(&bars->p_full[x]));
                ++n;
            } while (!(flags & kLast));
        } else {  // the other row tile's steps
            do {
                if (!wait(&bars->step[n % C::M], (uint32_t)(n / C::M), &bars->stop)) return;
                if (!wait(&bars->s_full[x], s_turn++, &bars->stop)) return;
                flags = steps[n % C::M].flags;
                __syncwarp();
                if (lane == 0) arrive(smem_of(&bars->p_full[x]));
                ++n;
            } while (!(flags & kLast));
        }
        // the next piece's queries while the last product runs: its scores are through
        more = walk.next(a, &p);
        if (more) load_q();
        if (valid > 0 || x == 0) {
            if (!wait(&bars->o_done[x], o_turn++, &bars->stop)) return;
            tc_after();
            if (busy) {
                drain();
                if (r < valid)
                    *reinterpret_cast<float2*>(part - (x * 128 + r) * 8 + ROWS * D + (x * 128 + r) * 2) =
                        make_float2(ref, l);
            }
        }
    }
}

template <class T, class C>
__global__ void __launch_bounds__(C::kThreads, 1) prefix_kernel(const PrefixArgs a) {
    extern __shared__ unsigned char raw[];
    __shared__ Bars bars;
    __shared__ Step steps[C::M];
    unsigned char* smem = raw + ((1024 - (smem_of(raw) & 1023)) & 1023);
    const int wp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::S; ++i) {
            rmsn::mbar_init(smem_of(&bars.k_full[i]), 4);
            rmsn::mbar_init(smem_of(&bars.v_full[i]), 4);
            rmsn::mbar_init(smem_of(&bars.k_free[i]), 1);
            rmsn::mbar_init(smem_of(&bars.v_free[i]), 1);
        }
        for (int i = 0; i < C::M; ++i) rmsn::mbar_init(smem_of(&bars.step[i]), 1);
        for (int i = 0; i < C::R; ++i) {
            rmsn::mbar_init(smem_of(&bars.s_full[i]), 1);
            rmsn::mbar_init(smem_of(&bars.p_full[i]), 4);
            rmsn::mbar_init(smem_of(&bars.q_full[i]), 4);
            rmsn::mbar_init(smem_of(&bars.o_done[i]), 1);
        }
        rmsn::mbar_init(smem_of(&bars.last), 1);
        bars.stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (wp == 4 * C::R + 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&bars.tmem)),
                     "n"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (wp < 4 * C::R) soften<T, C>(a, smem, &bars, steps, wp >> 2);
    else if (wp < 4 * C::R + 4) produce<C>(a, smem + C::R * C::kQ, &bars, steps, wp & 3);
    else multiply<C>(smem, &bars, steps);
    tc_before();
    __syncthreads();
    tc_after();
    if (wp == 4 * C::R + 4)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(bars.tmem), "n"(C::kCols) : "memory");
    if (threadIdx.x == 0 && bars.stop) atomicOr(a.status, kWaitRanOut);
}

template <class C>
PrefixEntry entry(int dt) {
    return PrefixEntry{dt, C::D, C::R, C::TOK, C::kThreads, C::kSmem,
                       dt == 1 ? (const void*)&prefix_kernel<BF16, C> : (const void*)&prefix_kernel<F16, C>};
}

}  // namespace prefix
}  // namespace rmsattn
