// Attention over the paged E4M3 cache: the kernels.
//
//   s_j = scale q . k_j,  m = max s_j,  out = sum exp(s_j - m) v_j / sum exp(s_j - m)
//
// in one pass over the tokens: m, the sum l and the weighted sum O are carried
// along, and multiplied by exp(m_old - m_new) where the maximum grows.
//
// What bounds it.  A decode step reads 2 D + 1/2 bytes per token and key head
// and does 4 D products for each of the G query heads that share it: DRAM, as
// long as the G n columns (query head x query token) of a row stay few.  Each
// token also costs instructions, about 20 a warp at head_dim 128 and one
// column tile (a conversion for every two codes, a third of them; then the
// copies, the softmax of eight columns, the matrix products).  168 registers
// leave 12 warps an SM; with half the bytes a token (head_dim 64) or twice the
// columns those no longer cover each other's fixed latencies, the first stall
// there, with 40 to 50 % of the issue slots in use: latency at low occupancy is
// then the bound.  On one GB300, of the copy peak of 6.78 TB/s: 64 sequences of
// 6144 to 8192 tokens, 32 / 8 heads x 128, 0.94 GB in 146 us (0.95); the same
// at head_dim 64, 80 us (0.87), at 256, 149 us for half as many (0.93); 4 query
// tokens, 16 columns, 176 MB in 47 us (0.55); one sequence of 131072 tokens
// 52 us (0.77).
// So the work is laid out around the reads:
//
// * Columns are the narrow side of mma.m16n8k16: S^T = K Q^T with 16 tokens
//   as its rows, O^T = V^T P^T with 16 dims as its rows.  The codes are
//   widened to fp16 (exact) on their way from shared memory into the operand
//   registers; tcgen05 would need 16-bit copies of the codes in shared memory
//   first, twice their traffic, for matrices of 8 columns.
// * A dot product may take its dims in any order, so a lane's 16-byte vector
//   of K covers four k-steps, and its 16-byte vectors of V (one for each of
//   its four tokens) cover all of its dims: only vector loads, and the swizzle
//   of the stage makes them free of bank conflicts.
// * P^T is turned from S^T's accumulator layout into the second product's
//   operand layout by movmatrix: no shared memory, and no exchange between
//   warps before a row ends.
// * Each warp streams its own steps (16 or 32 tokens) through its own ring of
//   cp.async stages, scales included, across row borders: no block barrier in
//   the stream.  K and V have two stages each, and each is filled again as
//   soon as it has been read (K before the softmax, V behind the second
//   product): with two stages, two steps are on their way.
// * Where its next 32 steps lie (page, place in the page, whether a mask
//   touches them) the warp's lanes work out together, one step each, a batch
//   ahead of its use.
// * Long rows: the steps of all rows (sequence x key head x column group) form
//   one line that the blocks of a resident grid share evenly, whatever the
//   lengths.  A row inside one block is finished there; the parts of a row
//   that a border cuts go to the workspace in fp32 and are joined, in block
//   order, by a second launch.
// * Short rows (a.split > 0): a cluster of a.split blocks takes one row, and
//   joins its parts through distributed shared memory: one launch, no
//   workspace, no scan of the lengths.
//   Either way nothing depends on timing.
#pragma once

#include "attn_common.cuh"

namespace rmsattn {

using rmsn::F2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kOpen = 1u << 12;  // of a tile's word: every query sees all of it
// A row's reference (what is taken from its scores before exp2) follows its
// maximum only when that has grown by more than 2^kSlack: a sum is then rarely
// rescaled twice.  Weights are thus up to 2^kSlack; they are multiplied by
// kLift before they are rounded to fp16, whose subnormals then end 2^-32 below
// the reference: what 2^17 tokens lose at most (2^-33 each) is 2^-16 of it.
// The values' scales stay out of the rounded weights: they may differ by any
// factor from tile to tile, and a weight would lose as many bits.  A tile's
// products are summed by themselves and enter the row's sum through an fp32
// multiply-add with the scale (16 packed ones a tile and column tile at
// head_dim 128).  Against weights times scale over the largest scale so far,
// which lost every bit at a ratio of 2^33: one column tile 38.4 / 40.2 us (256 x
// 300 tokens, no rescaling for scales), two 47.1 / 46.1 (48 x 2000), four 102 /
// 93.5 (the same with 8 queries).
constexpr float kNone = -3.402823466e38f;  // the reference before any token is seen
constexpr float kSlack = 7.f;
constexpr float kLift = 256.f;

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float exp2a(float x) {  // two ulp; exp2(-inf) = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held one row to four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN left out
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_over_rows(float v) {  // over lanes of equal lane % 4
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}
__device__ __forceinline__ float sum_over_rows(float v) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 16);
}
// High bit of each byte that holds an E4M3 NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// ---------------------------------------------------------------- shape

// D head dim; NT column tiles of 8; KT tiles of 16 tokens in a step; W warps;
// M blocks share an SM.
template <int D_, int NT_, int KT_, int W_, int M_>
struct Shape {
    static constexpr int D = D_, NT = NT_, KT = KT_, W = W_, M = M_;
    static constexpr int kTok = 16 * KT;           // tokens of a step
    static constexpr int kCols = 8 * NT;           // columns of a row
    static constexpr int kTile = 16 * D;           // bytes of 16 tokens of K or V
    static constexpr int kSide = KT * kTile;       // bytes of a step of K or V
    static constexpr int kWarp = 4 * kSide;        // a warp's ring: K, K, V, V
    static constexpr int kMeta = 16 * KT;          // a warp's: K scale and V scale of two steps' tiles
    static constexpr int kQPitch = 2 * D + 16;     // fp16 query row; + 16: no bank conflicts
    // fp32 of a tile of every warp: the join between the block's rows; the same
    // room takes a cluster's parts of the block's dims
    static constexpr int kJoin = W * 8 * D * 4;
    static_assert(W * 8 >= kCols, "a cluster's parts: D / split dims of all columns, split times");
    // the rings; behind the last step, the join of all columns
    static constexpr int kRing = W * kWarp > NT * kJoin ? W * kWarp : NT * kJoin;
    static constexpr int kMetaAll = W * kMeta;
    static constexpr int kQ = kCols * kQPitch;
    static constexpr int kSmem = kRing + kMetaAll + kQ + kJoin;
};

// ---------------------------------------------------------------- rows and steps

// What a sequence's rows see, in tokens and steps of TOK tokens.
template <int TOK>
struct Span {
    int L;      // tokens of the sequence
    int end;    // tokens within the table: [0, end)
    int lo;     // first token that any query's window reaches (0 without a window)
    int sink;   // tokens [0, sink) stay visible
    int n_sink; // steps before the gap (those of the sinks), or all of them
    int jump;   // step numbers from n_sink on are this much higher
    int ns;     // steps, at least 1

    // tokens are counted from `start` on (a multiple of 16)
    __device__ __forceinline__ void of(const AttendArgs& a, int len, int start = 0) {
        L = len < 0 ? 0 : len - start;
        const int room = (int)(a.table_width * a.c.page) - start;
        end = L < room ? L : room;
        lo = 0;
        sink = a.sinks < end ? a.sinks : end;
        const int all = (end + TOK - 1) / TOK;
        n_sink = all;
        jump = 0;
        ns = all;
        if (a.window > 0) {
            lo = L - a.n - a.window + 1;
            if (lo < 0) lo = 0;
            const int s = (sink + TOK - 1) / TOK, w = (lo < end ? lo : end) / TOK;
            if (w > s) {
                n_sink = s;
                jump = w - s;
                ns = all - jump;
            }
        }
        if (ns < 1) ns = 1;
    }
    // kOpen if every query sees all of the 16 tokens from j on
    __device__ __forceinline__ uint32_t open(const AttendArgs& a, int j) const {
        return j + 15 <= L - a.n && j + 16 <= end &&
                       (a.window == 0 || j > L - 1 - a.window || j + 16 <= sink)
                   ? kOpen
                   : 0u;
    }
    // which of the 16 tokens from j on some query sees
    __device__ __forceinline__ uint32_t rows(int j) const {
        auto below = [&](int x) { return x <= j ? 0u : (x - j >= 16 ? 0xFFFFu : (1u << (x - j)) - 1u); };
        return below(end) & (~below(lo) | below(sink)) & 0xFFFFu;
    }
    __device__ __forceinline__ int first_token(int step) const {
        return (step < n_sink ? step : step + jump) * TOK;
    }
};

// A place on the line of all steps: row (b, hc), its first step's place, and
// the row's steps.
struct Place {
    int64_t b;
    int64_t first;  // place of the row's first step
    int hc;
};

// Steps of all rows on the line, the size of a share, the place of the caller's
// own, and the row that holds it.
struct Line {
    int64_t total, chunk, at;  // at >= total: nothing there
    Place row;
};

__device__ __forceinline__ int64_t chunk_of(const AttendArgs& a, int64_t total) {
    const int64_t c = (total + a.shares - 1) / a.shares;
    return c < a.min_chunk ? a.min_chunk : c;
}

// First token of sequence b that is not in a shared prefix.
template <bool PRE>
__device__ __forceinline__ int start_of(const AttendArgs& a, int64_t b) {
    if constexpr (PRE) return a.seqs[b].start;
    else return 0;
}

// Every thread of the block calls this.  Sequences are scanned THREADS at a
// time; up to THREADS of them (any usual batch) are scanned once.
template <int TOK, int THREADS, bool PRE>
__device__ __forceinline__ void find_share(const AttendArgs& a, Line* line) {
    __shared__ int64_t sums[THREADS / 32], found[3];
    constexpr int NW = THREADS / 32;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t HC = (int64_t)a.c.H * a.groups;
    const bool once = a.B <= THREADS;
    line->at = INT64_MAX;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t carry = 0;  // steps of a key head and column group, of the sequences so far
        for (int64_t b0 = 0; b0 < a.B; b0 += THREADS) {
            const int64_t b = b0 + threadIdx.x;
            int64_t ns = 0;
            if (b < a.B) {
                Span<TOK> s;
                s.of(a, a.lengths[b], start_of<PRE>(a, b));
                ns = s.ns;
            }
            int64_t inc = ns;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) sums[wp] = inc;
            __syncthreads();
            int64_t before = carry;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const int64_t v = sums[w];
                if (w < wp) before += v;
                carry += v;
            }
            __syncthreads();
            if (once) {
                line->total = carry * HC;
                line->chunk = chunk_of(a, line->total);
                line->at = blockIdx.x * line->chunk;
            }
            const int64_t p0 = (before + inc - ns) * HC, p1 = (before + inc) * HC;
            if (b < a.B && line->at >= p0 && line->at < p1) {
                const int64_t hc = (line->at - p0) / ns;
                found[0] = b;
                found[1] = hc;
                found[2] = p0 + hc * ns;
            }
        }
        if (once) break;
        line->total = carry * HC;
        line->chunk = chunk_of(a, line->total);
        line->at = blockIdx.x * line->chunk;
        if (line->at >= line->total) break;
    }
    __syncthreads();
    line->row.b = found[0];
    line->row.hc = (int)found[1];
    line->row.first = found[2];
}

// ---------------------------------------------------------------- one row's results

// Column c (0 .. kCols - 1) of column group cg: its query token and head.
struct Col {
    int qi, head;
    bool on;
};
__device__ __forceinline__ Col column(const AttendArgs& a, int hk, int cg, int c, int cols) {
    const int cc = cg * cols + c;
    Col r;
    r.on = cc < a.cols;
    r.qi = (int)((uint64_t)(uint32_t)cc * a.group_rcp >> 32);  // cc / group
    r.head = (hk - r.qi) * a.group + cc;
    return r;
}

template <class T>
__device__ __forceinline__ void store8(const AttendArgs& a, int64_t b, const Col& c, int d,
                                       const float (&y)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = rmsn::pack2<T>(y[2 * i], y[2 * i + 1]);
    uint16_t* o = static_cast<uint16_t*>(a.out) + (b * a.n + c.qi) * a.out_stride +
                  (int64_t)c.head * a.c.D + d;
    *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void add8(float (&y)[8], const float4* p, float f) {
    const float4 u = p[0], v = p[1];
    y[0] += u.x * f;
    y[1] += u.y * f;
    y[2] += u.z * f;
    y[3] += u.w * f;
    y[4] += v.x * f;
    y[5] += v.y * f;
    y[6] += v.z * f;
    y[7] += v.w * f;
}
// The four-float unit that holds dim d of a join row: the lanes that write a
// row's units 4 or 2 apart, and those that read it, meet different banks.
__device__ __forceinline__ int unit_at(int d) {
    const int u = d >> 2;
    return (u ^ ((u >> 3) & 3)) << 2;
}
__device__ __forceinline__ void read8(float4 (&v)[2], const float* row, int d) {
    v[0] = *reinterpret_cast<const float4*>(row + unit_at(d));
    v[1] = *reinterpret_cast<const float4*>(row + unit_at(d + 4));
}
// Eight dims of a row's sums over its weights' sum; nothing seen gives 0.  PRE: the
// sums as they are, with reference mx, for the join with the shared prefix's.
template <class T, bool PRE>
__device__ __forceinline__ void finish8(const AttendArgs& a, int64_t b, const Col& c, int d, float (&y)[8],
                                        float l, float mx) {
    if constexpr (PRE) {
        const int64_t row = (b * a.n + c.qi) * a.Hq + c.head;
        float4* o = reinterpret_cast<float4*>(a.own + row * a.c.D + d);
        o[0] = make_float4(y[0], y[1], y[2], y[3]);
        o[1] = make_float4(y[4], y[5], y[6], y[7]);
        if (d == 0) a.own_ml[row] = make_float2(mx, l);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = l == 0.f ? 0.f : y[k] / l;
    store8<T>(a, b, c, d, y);
}

// ---------------------------------------------------------------- the cluster's shared memory

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_begin() {  // arrives; orders no memory
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, int rank, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(in_block(addr, rank)), "f"(v.x),
                 "f"(v.y)
                 : "memory");
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, int rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(in_block(addr, rank)),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// The workspace: a Cut for every share, then two parts for every share.
// Share i's Cut tells of the row that its upper border cuts, if i is the first
// share that the row lies in: whose it is, which of share i's parts is its
// first, and the last share it reaches.  Every share writes its Cut.
struct __align__(16) Cut {
    int64_t b;
    int64_t last;
    int32_t hc;
    int32_t which;
    int32_t on;
    int32_t pad;
};
static_assert(sizeof(Cut) == kCutBytes, "the workspace is sized on the host");
__device__ __forceinline__ Cut* cut_of(const AttendArgs& a, int64_t blk) {
    return reinterpret_cast<Cut*>(a.ws) + blk;
}
// Partial results of share `blk`'s first (0) or last (1) row.
template <class C>
__device__ __forceinline__ float* part_of(const AttendArgs& a, int64_t blk, int which) {
    return reinterpret_cast<float*>(a.ws + a.shares * kCutBytes) +
           (blk * 2 + which) * (int64_t)(C::kCols * (C::D + 2));
}

// ---------------------------------------------------------------- the stream

// One tile's weighted values, token by token, for the columns that see each
// (the values' NaN reaches those alone).  p: the packed weights as the scores
// lie: tokens g and g + 8, columns 2 t and 2 t + 1; see: their bits; f: the
// tile's value scale.  A path for NaN codes under a mask only: small rather
// than fast.
template <class C>
__device__ __forceinline__ void add_tile(F2 (&o)[C::D / 16][C::NT][2], const uint32_t (&p)[C::NT][2],
                                         uint32_t see, uint32_t vt, float f) {
    constexpr int D = C::D, MT = D / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 1
    for (int r = 0; r < 16; ++r) {
        const int from = (r & 7) * 4 + t, h = r >> 3;
        const uint32_t bits = __shfl_sync(0xFFFFFFFFu, see, from) >> (2 * h);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
            const uint32_t w0 = __shfl_sync(0xFFFFFFFFu, p[nt][0], from);
            const uint32_t w1 = __shfl_sync(0xFFFFFFFFu, p[nt][1], from);
            const uint32_t w = h ? w1 : w0;
            // weights of 0, and values of 0 beside them, where a column sees nothing
            const bool on0 = bits >> (4 * nt) & 1, on1 = bits >> (4 * nt + 1) & 1;
            const float p0 = rmsn::lo2<F16>(w) * f, p1 = rmsn::hi2<F16>(w) * f;
#pragma unroll
            for (int i = 0; i < MT; ++i) {  // dims 2 i and 2 i + 1 of the lane's
                const int d = D == 64 ? g * 8 + 2 * i : (g + 8 * (i / 8)) * 16 + 2 * (i % 8);
                const int e = r * (D / 16) + d / 16;  // 16-byte chunk, swizzled as V is
                const int at = D == 64 ? (e & ~7) + ((e & 7) ^ (((r >> 1) & 3) * 2)) : e ^ (((r >> 1) & 3) * 2);
                uint16_t v;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(vt + at * 16 + d % 16) : "memory");
                const uint32_t x = e4m3x2_to_f16x2(v);
                const float v0 = rmsn::lo2<F16>(x), v1 = rmsn::hi2<F16>(x);
                const F2 pp = rmsn::f2(p0, p1);
                o[i][nt][0] = rmsn::fma2(rmsn::f2(on0 ? v0 : 0.f, on1 ? v0 : 0.f), pp, o[i][nt][0]);
                o[i][nt][1] = rmsn::fma2(rmsn::f2(on0 ? v1 : 0.f, on1 ? v1 : 0.f), pp, o[i][nt][1]);
            }
        }
    }
}

// A block's warps take the steps of its share in turn, and are joined where a
// row ends.
template <class T, class C, bool PRE = false>
__global__ void __launch_bounds__(C::W * 32, C::M) attend_kernel(const AttendArgs a) {
    constexpr int D = C::D, NT = C::NT, KT = C::KT, W = C::W;
    constexpr int CH = D / 16;                 // 16-byte chunks of a token
    constexpr int MT = D / 16;                 // tiles of 16 dims
    constexpr bool kQRegs = NT == 1 && D <= 128 && KT == 1;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float q_scale[C::kCols];
    __shared__ int q_index[C::kCols];  // a column's query token
    __shared__ float2 part_ml[kMaxSplit][C::kCols];  // references and sums of a cluster's blocks
    __shared__ float j_m[W][C::kCols], j_l[W][C::kCols];
    rmsn::pdl_wait(a.pdl);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    // a block's shared memory may be written to once the block has begun
    if (a.split > 1) cluster_begin();

    // this share's steps: `count` from place `begin`, the first of them in row
    // `at` (whose first step lies at at.first <= begin)
    int64_t begin, chunk = 0;
    int count;
    Place at;
    if (a.split > 0) {
        const uint32_t HC = (uint32_t)(a.c.H * a.groups), row = blockIdx.x >> a.split_log;
        at.b = row / HC;
        at.hc = (int)(row % HC);
        at.first = 0;
        Span<C::kTok> s;
        s.of(a, a.lengths[at.b], start_of<PRE>(a, at.b));
        const int per = (s.ns + a.split - 1) >> a.split_log;
        begin = (int64_t)((int)blockIdx.x & (a.split - 1)) * per;
        const int left = s.ns - (int)begin;
        count = left < 0 ? 0 : (left < per ? left : per);
    } else {
        Line line;
        find_share<C::kTok, W * 32, PRE>(a, &line);
        begin = line.at;
        chunk = line.chunk;
        at = line.row;
        if (begin >= line.total) {
            if (threadIdx.x == 0) cut_of(a, blockIdx.x)->on = 0;
            return;
        }
        count = (int)(line.total - begin < chunk ? line.total - begin : chunk);
    }

    unsigned char* qrows = smem + C::kRing + C::kMetaAll;
    const uint32_t ring_s = smem_addr(smem) + wp * C::kWarp, meta_s = smem_addr(smem) + C::kRing + wp * C::kMeta;

    // ---- queries: this warp's columns of a row, first into registers (before
    // the wait that they can hide behind), then to shared memory in fp16, each
    // scaled by a power of two to at most 2^8 (so that fp16 holds any bf16 row:
    // each element exactly, or to within 2^-32 of the row's largest, half of
    // the subnormals' step over 2^7); q_scale undoes it, times |scale| log2(e)
    // (a negative scale turns the queries' sign)
    constexpr int QC = (C::kCols + W - 1) / W, QW = D / 64;
    uint32_t qreg[QC][QW];
    auto load_q = [&](int64_t b, int hc) {
        const int hk = hc / a.groups, cg = hc % a.groups;
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const Col col = column(a, hk, cg, wp + i * W, C::kCols);
            const uint16_t* p = static_cast<const uint16_t*>(a.q) + (b * a.n + col.qi) * a.q_stride +
                                (int64_t)col.head * D + 2 * lane;
#pragma unroll
            for (int k = 0; k < QW; ++k)
                qreg[i][k] = col.on && wp + i * W < C::kCols
                                 ? *reinterpret_cast<const uint32_t*>(p + 64 * k)
                                 : 0u;
        }
    };
    auto store_q = [&](int cg) {
        for (int c = threadIdx.x; c < C::kCols; c += W * 32)
            q_index[c] = column(a, 0, cg, c, C::kCols).qi;
#pragma unroll
        for (int i = 0; i < QC; ++i) {
            const int c = wp + i * W;
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < QW; ++k)
                m = rmsn::absmax3(m, rmsn::lo2<T>(qreg[i][k]), rmsn::hi2<T>(qreg[i][k]));
            m = rmsn::warp_max(m);
            int e = (int)(__float_as_uint(m) >> 23) - 127 - 7;  // 2^e <= m / 128 < 2^(e + 1)
            e = e < -126 ? -126 : (e > 126 ? 126 : e);
            // an infinite element makes every score of the row infinite or NaN,
            // and any softmax of such scores NaN (all of -inf among them)
            const float down = m > 3.402823466e38f
                                   ? __uint_as_float(0x7FFFFFFFu)
                                   : copysignf(__uint_as_float((uint32_t)(127 - e) << 23), a.scale);
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
            if (c >= C::kCols) break;
            if (lane == 0) q_scale[c] = up * (fabsf(a.scale) * kLog2e);
#pragma unroll
            for (int k = 0; k < QW; ++k)
                *reinterpret_cast<uint32_t*>(qrows + c * C::kQPitch + (64 * k + 2 * lane) * 2) =
                    rmsn::pack_f16x2(rmsn::lo2<T>(qreg[i][k]) * down, rmsn::hi2<T>(qreg[i][k]) * down);
        }
    };
    load_q(at.b, at.hc);

    // ---- producer: this warp's steps of the share's `count`
    //
    // A batch: up to 32 of the warp's steps of one row, one to a lane; `next_`
    // is on its way (its table entries are loading) while the other is used.
    // A tile's word: its block of 16 tokens in the page (12 bits), whether every
    // query sees all of it (bit 12), and from bit 16 on which of its rows some
    // query sees (none where the page is bad).
    int p_at = wp, p_first = (int)(at.first - begin), p_hc = at.hc;  // places relative to begin
    int64_t p_b = at.b;
    Span<C::kTok> p_span;
    int p_start = start_of<PRE>(a, p_b), p_start_next = 0;
    p_span.of(a, a.lengths[p_b], p_start);
    int p_len_next = 0;
    if (p_b + 1 < a.B) {
        p_len_next = a.lengths[p_b + 1];
        p_start_next = start_of<PRE>(a, p_b + 1);
    }
    const int32_t* p_row = a.table + p_b * a.table_stride;
    int b_n = 0, b_at = 0, next_n = 0, next_hk = 0;
    int32_t next_page[KT];
    uint32_t b_where[KT], next_where[KT];
    int64_t b_off[KT];   // bytes from the cache's begin to the tile
    uint32_t b_scale[KT];  // the tile's scale, counted from the first
    auto look_ahead = [&]() {
        next_n = 0;
        if (p_at >= count) return;
        while (p_at >= p_first + p_span.ns) {
            p_first += p_span.ns;
            if (++p_hc == a.c.H * a.groups) {
                p_hc = 0;
                ++p_b;
                p_row += a.table_stride;
                p_start = p_start_next;
                p_span.of(a, p_len_next, p_start);
                if (p_b + 1 < a.B) {
                    p_len_next = a.lengths[p_b + 1];
                    p_start_next = start_of<PRE>(a, p_b + 1);
                }
            }
        }
        const int end = p_first + p_span.ns < count ? p_first + p_span.ns : count;
        next_n = (end - p_at + W - 1) / W;
        if (next_n > 32) next_n = 32;
        next_hk = p_hc / a.groups;
        const int t0 = p_span.first_token(p_at + lane * W - p_first);
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const int j = t0 + 16 * k;
            const bool any = lane < next_n && j < p_span.end && (j + 15 >= p_span.lo || j < p_span.sink);
            // slot = j / page, both multiples of 16: exact for j < 2^29
            const int at = PRE ? j + p_start : j;
            const int slot = (int)(((uint64_t)(uint32_t)(at >> 4) * a.page_rcp) >> 37);
            next_page[k] = any ? p_row[slot] : -1;  // end lies within the table
            next_where[k] = (uint32_t)((at - slot * a.c.page) >> 4) |
                            (any ? p_span.open(a, j) | (p_span.rows(j) << 16) : 0u);
        }
        p_at += next_n * W;
    };
    auto turn_page = [&]() {  // the batch that was on its way becomes the one in use
        b_n = next_n;
        b_at = 0;
        if (next_n == 0) return;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            b_where[k] = next_where[k];
            int64_t page = next_page[k];
            if ((uint32_t)next_page[k] >= (uint32_t)a.c.n_pages) {
                if (b_where[k] >> 16) atomicOr(a.status, kBadPage);
                page = 0;
                b_where[k] = 0;
            }
            const int tile = next_hk * (a.c.page >> 4) + (int)(b_where[k] & 0xFFF);
            b_off[k] = page * a.c.page_stride + (int64_t)tile * C::kTile;
            b_scale[k] = (uint32_t)(page * a.c.scale_stride) + (uint32_t)tile;
        }
        look_ahead();
    };
    // Lane constants of the copies: chunk i of a tile is 512 i bytes on in
    // memory, and in the stage too, but for V's swizzle, which flips with i.
    const int l_row = lane / CH, l_chunk = lane % CH;
    uint32_t k_dst, v_dst[2];
    if constexpr (D == 64) {  // two tokens to a 128-byte line, 8 tokens a copy
        k_dst = lane * 16;
        v_dst[0] = v_dst[1] = ((lane & ~7) + ((lane & 7) ^ (((l_row >> 1) & 3) * 2))) * 16;
    } else if constexpr (D == 128) {  // 4 tokens a copy
        k_dst = (l_row * CH + (l_chunk ^ ((l_row & 1) * 4))) * 16;
        v_dst[0] = (l_row * CH + (l_chunk ^ ((l_row >> 1) * 2))) * 16;
        v_dst[1] = (l_row * CH + (l_chunk ^ (((l_row >> 1) * 2) ^ 4))) * 16;
    } else {  // 2 tokens a copy
        k_dst = (l_row * CH + (l_chunk ^ (l_row * 4))) * 16;
        v_dst[0] = v_dst[1] = lane * 16;  // and the swizzle (i & 3) * 2, below
    }
    auto v_at = [&](int i) -> uint32_t {
        if constexpr (D == 256) return v_dst[0] ^ ((i & 3) * 32);
        else return v_dst[i & 1];
    };
    // the step to copy: its tiles' places and states
    bool s_on = false;
    uint32_t s_where[KT], s_scale[KT];
    int64_t s_off[KT];
    auto locate = [&]() {
        if (b_at == b_n) turn_page();
        s_on = b_at < b_n;
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            s_off[k] = __shfl_sync(0xFFFFFFFFu, b_off[k], b_at);
            s_scale[k] = __shfl_sync(0xFFFFFFFFu, b_scale[k], b_at);
            s_where[k] = s_on ? __shfl_sync(0xFFFFFFFFu, b_where[k], b_at) : 0u;
        }
        ++b_at;
    };
    // this lane's 16 bytes of a tile; lanes 2 k and 2 k + 1 copy tile k's scales
    const uint8_t *k_src = a.c.k + lane * 16, *v_src = a.c.v + lane * 16;
    const float* scale_src = (lane & 1) ? a.c.vs : a.c.ks;
    auto copy_step = [&](uint32_t dst, const uint8_t* base, bool v) {
        bool open = true;
#pragma unroll
        for (int k = 0; k < KT; ++k) open = open && (s_where[k] & kOpen);
        if (open) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    cp16(dst + k * C::kTile + (v ? v_at(i) : k_dst) + i * 512, base + s_off[k] + i * 512);
        } else if (s_on) {  // rows that no query sees are zeros
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    cp16(dst + k * C::kTile + (v ? v_at(i) : k_dst) + i * 512, base + s_off[k] + i * 512,
                         s_where[k] >> (16 + l_row + i * (32 / CH)) & 1);
        }
    };
    // the located step's K and scales, or V, into stage `slot`
    auto issue_k = [&](int slot) {
        copy_step(ring_s + slot * C::kSide, k_src, false);
        uint32_t at = s_scale[0], rows = s_where[0];
#pragma unroll
        for (int k = 1; k < KT; ++k)
            if (lane >> 1 == k) {
                at = s_scale[k];
                rows = s_where[k];
            }
        if (lane < 2 * KT && rows >> 16)
            cp4(meta_s + slot * (8 * KT) + lane * 4, scale_src + at);
        cp_commit();
    };
    auto issue_v = [&](int slot) {
        copy_step(ring_s + (2 + slot) * C::kSide, v_src, true);
        cp_commit();
    };

    uint32_t where[2][KT];  // tiles of the step in work and of the next
    look_ahead();
    turn_page();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        locate();
        issue_k(i);
        issue_v(i);
#pragma unroll
        for (int k = 0; k < KT; ++k) where[i][k] = s_where[k];
    }
    locate();

    // ---- consumer: rows one after another, this warp's steps of each
    int slot = 0;
    int cur = 0;  // the row's first place within this share
    int mine = wp;
    int64_t c_b = at.b;
    int c_first = (int)(at.first - begin), c_hc = at.hc;
    Span<C::kTok> span;
    span.of(a, a.lengths[c_b], start_of<PRE>(a, c_b));
    int c_len_next = 0, c_start_next = 0;
    if (c_b + 1 < a.B) {
        c_len_next = a.lengths[c_b + 1];
        c_start_next = start_of<PRE>(a, c_b + 1);
    }
    do {  // once at least: a block of a cluster may have no steps
        const int row_end = c_first + span.ns;
        // (a cluster's block works on one row, and may lie behind its end)
        const int seg_end = a.split == 0 && row_end < count ? row_end : count;
        const int hk = c_hc / a.groups, cg = c_hc % a.groups;
        if (span.L > span.end && threadIdx.x == 0) atomicOr(a.status, kBadPage);

        store_q(cg);
        __syncthreads();
        F2 cs[NT];  // the lane's two columns of each tile, here and below
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            cs[nt] = rmsn::f2(q_scale[nt * 8 + 2 * t], q_scale[nt * 8 + 2 * t + 1]);
        const uint32_t q_s = smem_addr(qrows) + g * C::kQPitch + t * 32;
        uint4 qf[kQRegs ? CH / 2 : 1];
        if constexpr (kQRegs) {
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) qf[i] = lds16(q_s + (i / 2) * 128 + (i & 1) * 16);
        }
        F2 o[MT][NT][2];  // two columns each, of two dims
        F2 less[NT], l[NT];  // minus the references; the weights' sums
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            less[nt] = rmsn::f2(-kNone, -kNone);
            l[nt] = rmsn::f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) o[i][nt][k] = rmsn::f2(0.f, 0.f);
        }

        for (; mine < seg_end; mine += W) {
            cp_wait<3>();  // K and the scales; behind them V, and the next step's both
            __syncwarp();
            float ks[KT], vs[KT];
            bool open = true;  // no mask touches this step
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const uint2 sc = lds8(meta_s + slot * (8 * KT) + k * 8);
                ks[k] = __uint_as_float(sc.x);
                vs[k] = __uint_as_float(sc.y);
                open = open && (where[0][k] & kOpen);
            }
            if (!open) {  // a tile that brought nothing in left an older scale
#pragma unroll
                for (int k = 0; k < KT; ++k)
                    if (!(where[0][k] >> 16)) ks[k] = vs[k] = 0.f;
            }
            const uint32_t st = ring_s + slot * C::kSide;

            // S^T = K Q^T
            float s[KT][NT][4];
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[k][nt][x] = 0.f;
#pragma unroll
            for (int j = 0; j < CH / 4; ++j) {
                uint4 qa[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (kQRegs) qa[nt][h] = qf[2 * j + h];
                        else qa[nt][h] = lds16(q_s + nt * 8 * C::kQPitch + j * 128 + h * 16);
                    }
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    const int c = D == 64 ? t : ((t + 4 * j) ^ ((g & 1) * 4));
                    const uint4 k0 = lds16(st + k * C::kTile + (g * CH + c) * 16);
                    const uint4 k1 = lds16(st + k * C::kTile + ((g + 8) * CH + c) * 16);
                    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t a0 = e4m3x2_to_f16x2(w0[u]), a2 = e4m3x2_to_f16x2(w0[u] >> 16);
                        const uint32_t a1 = e4m3x2_to_f16x2(w1[u]), a3 = e4m3x2_to_f16x2(w1[u] >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 q = qa[nt][u >> 1];
                            mma16816(s[k][nt], a0, a1, a2, a3, (u & 1) ? q.z : q.x, (u & 1) ? q.w : q.y);
                        }
                    }
                }
            }

            __syncwarp();
            issue_k(slot);  // every lane has read this stage

            // Exponents are S kc - m in units of log2, kc = K scale x query
            // scale (not negative).  A mask makes S -inf, and the weight 0 below.
            uint32_t see[KT];  // bit 4 nt + x: this lane's element is visible
            if (!open) {
                const int t0 = span.first_token(mine - c_first);
#pragma unroll
                for (int k = 0; k < KT; ++k) see[k] = 0u;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int pos = span.L - a.n + q_index[nt * 8 + 2 * t + x];
                        const int from = a.window == 0 ? 0 : pos - a.window + 1;
#pragma unroll
                        for (int k = 0; k < KT; ++k)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int j = t0 + 16 * k + g + 8 * h;
                                const bool on = (where[0][k] >> (16 + g + 8 * h) & 1) && j <= pos &&
                                                (j >= from || j < a.sinks);
                                if (on) see[k] |= 1u << (4 * nt + 2 * h + x);
                                else s[k][nt][2 * h + x] = -INFINITY;
                            }
                    }
            }
            F2 kc[KT][NT], e[KT][NT][2];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < KT; ++k) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    kc[k][nt] = rmsn::mul2(rmsn::f2(ks[k], ks[k]), cs[nt]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float lo, hi;
                        e[k][nt][h] = rmsn::fma2(rmsn::f2(s[k][nt][2 * h], s[k][nt][2 * h + 1]), kc[k][nt], less[nt]);
                        rmsn::f2split(e[k][nt][h], lo, hi);
                        top = max3(top, lo, hi);
                    }
                }
            }
            if (__any_sync(0xFFFFFFFFu, top > kSlack)) {
                // new references; what was summed so far follows them
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float to[2], was[2], keep[2];
                    rmsn::f2split(less[nt], was[0], was[1]);
                    to[0] = -was[0];
                    to[1] = -was[1];
#pragma unroll
                    for (int k = 0; k < KT; ++k) {
                        float c[2];
                        rmsn::f2split(kc[k][nt], c[0], c[1]);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            to[x] = max3(to[x], __fmul_rn(s[k][nt][x], c[x]), __fmul_rn(s[k][nt][2 + x], c[x]));
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        to[x] = max_over_rows(to[x]);
                        keep[x] = exp2a(-was[x] - to[x]);
                    }
                    less[nt] = rmsn::f2(-to[0], -to[1]);
                    const F2 keep2 = rmsn::f2(keep[0], keep[1]);
                    l[nt] = rmsn::mul2(l[nt], keep2);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) o[i][nt][x] = rmsn::mul2(o[i][nt][x], keep2);
                    // from the rounded products, as the reference was taken: the
                    // largest then weighs 1 where scores are beyond 2^28, too
                    // (what a product rounds off there is a large exponent); one
                    // by one, for the compiler contracts the packed forms
#pragma unroll
                    for (int k = 0; k < KT; ++k) {
                        float c[2];
                        rmsn::f2split(kc[k][nt], c[0], c[1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            e[k][nt][h] = rmsn::f2(__fsub_rn(__fmul_rn(s[k][nt][2 * h], c[0]), to[0]),
                                                   __fsub_rn(__fmul_rn(s[k][nt][2 * h + 1], c[1]), to[1]));
                    }
                }
            }

            // weights; P^T as the second product's operand
            uint32_t pb[KT][NT][2];
            float p[KT][NT][4];
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float lo, hi;
                        rmsn::f2split(e[k][nt][h], lo, hi);
                        p[k][nt][2 * h] = exp2a(lo);
                        p[k][nt][2 * h + 1] = exp2a(hi);
                    }
            if (!open) {
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (!(see[k] >> (4 * nt + x) & 1)) p[k][nt][x] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const F2 lift = rmsn::f2(kLift, kLift);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const F2 w = rmsn::f2(p[k][nt][2 * h], p[k][nt][2 * h + 1]);
                        float lo, hi;
                        l[nt] = rmsn::add2(l[nt], w);
                        rmsn::f2split(rmsn::mul2(w, lift), lo, hi);
                        pb[k][nt][h] = rmsn::pack_f16x2(lo, hi);
                    }
            }

            // O^T += V^T P^T
            cp_wait<3>();  // V; behind it the next step's K and V, and the K after
            __syncwarp();
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const uint32_t vt = st + 2 * C::kSide + k * C::kTile;
                // A token that some columns see and others do not may hold NaN
                // codes, which weights of 0 would carry into the others' sums:
                // then the tile is added token by token, where it is seen.
                bool nan = false;
                if (!open && a.n > 1) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint4 v = lds16(vt + lane * 16 + i * 512);
                        nan = nan || (nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w));
                    }
                    nan = __any_sync(0xFFFFFFFFu, nan);
                }
                // O's unit is 1: the scale takes the lift back (it stays exact
                // down to 2^-118; below, it keeps 16 bits)
                const float f = vs[k] * (1.f / kLift);
                if (nan) {
                    add_tile<C>(o, pb[k], see[k], vt, f);
                    continue;
                }
                const F2 f2 = rmsn::f2(f, f);
                uint32_t pt[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    pt[nt][0] = transpose8(pb[k][nt][0]);
                    pt[nt][1] = transpose8(pb[k][nt][1]);
                }
#pragma unroll
                for (int cj = 0; cj < (D == 256 ? 2 : 1); ++cj) {
                    constexpr int WD = D == 64 ? 2 : 4;  // words of dims a lane holds per token
                    uint32_t w[4][WD];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int r = 2 * t + (x & 1) + 8 * (x >> 1);
                        if constexpr (D == 64) {
                            const int e = r * 4 + (g >> 1);
                            const uint2 v = lds8(vt + ((e & ~7) + ((e & 7) ^ (2 * t))) * 16 + (g & 1) * 8);
                            w[x][0] = v.x;
                            w[x][1] = v.y;
                        } else {
                            const uint4 v = lds16(vt + (r * CH + ((g + 8 * cj) ^ (2 * t))) * 16);
                            w[x][0] = v.x;
                            w[x][1] = v.y;
                            w[x][2] = v.z;
                            w[x][3] = v.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < WD; ++i) {
                        const uint32_t lo01 = __byte_perm(w[0][i], w[1][i], 0x5140);
                        const uint32_t hi01 = __byte_perm(w[0][i], w[1][i], 0x7362);
                        const uint32_t lo23 = __byte_perm(w[2][i], w[3][i], 0x5140);
                        const uint32_t hi23 = __byte_perm(w[2][i], w[3][i], 0x7362);
                        const uint32_t a0 = e4m3x2_to_f16x2(lo01), a1 = e4m3x2_to_f16x2(lo01 >> 16);
                        const uint32_t a2 = e4m3x2_to_f16x2(lo23), a3 = e4m3x2_to_f16x2(lo23 >> 16);
                        const uint32_t b0 = e4m3x2_to_f16x2(hi01), b1 = e4m3x2_to_f16x2(hi01 >> 16);
                        const uint32_t b2 = e4m3x2_to_f16x2(hi23), b3 = e4m3x2_to_f16x2(hi23 >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float u[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                            mma16816(u[0], a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
                            mma16816(u[1], b0, b1, b2, b3, pt[nt][0], pt[nt][1]);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                F2& y = o[cj * 8 + 2 * i + (x >> 1)][nt][x & 1];
                                y = rmsn::fma2(rmsn::f2(u[x >> 1][2 * (x & 1)], u[x >> 1][2 * (x & 1) + 1]), f2, y);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            issue_v(slot);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                where[0][k] = where[1][k];
                where[1][k] = s_where[k];
            }
            locate();
            slot ^= 1;
        }

        const bool last = seg_end >= count;
        const bool whole = a.split > 0 ? a.split == 1 : cur == c_first && seg_end == row_end;
        float* part = part_of<C>(a, blockIdx.x, cur == 0 ? 0 : 1);
        if (threadIdx.x == 0 && last && a.split == 0) {
            Cut* cut = cut_of(a, blockIdx.x);
            cut->on = row_end > count && c_first >= 0;
            cut->b = c_b;
            cut->hc = c_hc;
            cut->which = cur == 0 ? 0 : 1;
            cut->last = (begin + row_end - 1) / chunk;
        }
        // the next row's queries and length, while this one is finished
        const int64_t row_b = c_b;
        if (!last) {
            if (++c_hc == a.c.H * a.groups) {
                c_hc = 0;
                ++c_b;
            }
            load_q(c_b, c_hc);
        }
        int used = a.cols - cg * C::kCols;  // columns of this row
        if (used > C::kCols) used = C::kCols;
        float ls[NT][2], m[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            rmsn::f2split(l[nt], ls[nt][0], ls[nt][1]);
            rmsn::f2split(less[nt], m[nt][0], m[nt][1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                ls[nt][x] = sum_over_rows(ls[nt][x]);
                m[nt][x] = -m[nt][x];
            }
        }
        // join the warps, a tile of eight columns at a time; behind the block's
        // last step the ring is free, and holds all of them
        const int tiles = (used + 7) / 8, step = last ? NT : 1;
        if (a.split > 1) cluster_wait();
        float* parts = reinterpret_cast<float*>(smem + C::kRing + C::kMetaAll + C::kQ);  // of a cluster
        float* join = reinterpret_cast<float*>(last ? smem : smem + C::kRing + C::kMetaAll + C::kQ);
        if (last) __syncthreads();  // every warp is through with its stages
        for (int n0 = 0; n0 < tiles; n0 += step) {
            if (n0 > 0) __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt < n0 || nt >= n0 + step) continue;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int cc = nt * 8 + 2 * t + x;
                    if (cc >= used) continue;
                    if (g == 0) {
                        j_m[wp][cc] = m[nt][x];
                        j_l[wp][cc] = ls[nt][x];
                    }
                    float* jr = join + ((cc - n0 * 8) * W + wp) * D;
#pragma unroll
                    for (int i = 0; i < MT; i += 2) {
                        const int d = D == 64 ? g * 8 + 2 * i : (g + 8 * (i / 8)) * 16 + 2 * (i % 8);
                        float y[4][2];  // dims d to d + 3 of both columns
                        rmsn::f2split(o[i][nt][0], y[0][0], y[0][1]);
                        rmsn::f2split(o[i][nt][1], y[1][0], y[1][1]);
                        rmsn::f2split(o[i + 1][nt][0], y[2][0], y[2][1]);
                        rmsn::f2split(o[i + 1][nt][1], y[3][0], y[3][1]);
                        *reinterpret_cast<float4*>(jr + unit_at(d)) =
                            make_float4(y[0][x], y[1][x], y[2][x], y[3][x]);
                    }
                }
            }
            __syncthreads();
            const int in = (used - n0 * 8 < step * 8 ? used - n0 * 8 : step * 8) * (D / 8);
            for (int e = threadIdx.x; e < in; e += W * 32) {  // columns x D / 8 vectors
                const int c = e / (D / 8), d = e % (D / 8) * 8, cc = n0 * 8 + c;
                const Col col = column(a, hk, cg, cc, C::kCols);
                float mx = kNone;
#pragma unroll
                for (int w = 0; w < W; ++w) mx = fmaxf(mx, j_m[w][cc]);
                float lsum = 0.f, y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float f = exp2a(j_m[w][cc] - mx);
                    lsum += j_l[w][cc] * f;
                    float4 v[2];
                    read8(v, join + (c * W + w) * D, d);
                    add8(y, v, f);
                }
                if (whole) {
                    finish8<T, PRE>(a, row_b, col, d, y, lsum, mx);
                } else if (a.split > 0) {
                    // to the block that finishes these dims, each sender its place
                    const int rank = (int)blockIdx.x & (a.split - 1);
                    const int item = cc * (D / 8) + d / 8, owner = item & (a.split - 1);
                    const uint32_t at = smem_addr(parts) + (item - owner + rank) * 32;
                    st_cluster4(at, owner, make_float4(y[0], y[1], y[2], y[3]));
                    st_cluster4(at + 16, owner, make_float4(y[4], y[5], y[6], y[7]));
                    if (d == 0)
                        for (int r = 0; r < a.split; ++r)
                            st_cluster2(smem_addr(&part_ml[rank][cc]), r, make_float2(mx, lsum));
                } else {
                    float4* dst = reinterpret_cast<float4*>(part + cc * D + d);
                    dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                    dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                    if (d == 0)
                        *reinterpret_cast<float2*>(part + C::kCols * D + cc * 2) =
                            make_float2(mx, lsum);
                }
            }
        }
        if (a.split > 1) {
            // every block's parts have arrived; nothing is sent behind this, so
            // a block may leave once it has read its own
            cluster_arrive();
            cluster_wait();
            const int rank = (int)blockIdx.x & (a.split - 1), items = used * (D / 8);
            for (int i = threadIdx.x; i * a.split + rank < items; i += W * 32) {
                const int item = i * a.split + rank, cc = item / (D / 8), d = item % (D / 8) * 8;
                const Col col = column(a, hk, cg, cc, C::kCols);
                const float4* from = reinterpret_cast<const float4*>(parts + i * a.split * 8);
                float mx = kNone, lsum = 0.f, y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = 0.f;
                float2 ml[kMaxSplit];
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r) {
                    ml[r] = r < a.split ? part_ml[r][cc] : make_float2(kNone, 0.f);
                    mx = fmaxf(mx, ml[r].x);
                }
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r) {
                    if (r >= a.split) break;
                    const float f = exp2a(ml[r].x - mx);
                    lsum += ml[r].y * f;
                    add8(y, from + 2 * r, f);
                }
                finish8<T, PRE>(a, row_b, col, d, y, lsum, mx);
            }
        }
        cur = seg_end;
        if (!last) {
            c_first = row_end;
            if (c_b != row_b) {
                span.of(a, c_len_next, c_start_next);
                if (c_b + 1 < a.B) {
                    c_len_next = a.lengths[c_b + 1];
                    c_start_next = start_of<PRE>(a, c_b + 1);
                }
            }
        }
    } while (cur < count);
    cp_wait<0>();
}

// Joins the parts of the rows that the shares' borders cut, in the shares'
// order.  Block (i, q): the row of share i's Cut, columns 4 q to 4 q + 3; D
// threads to a part (four dims of a column each), blockDim / D groups of them
// that take the parts in turn.  A thread takes up to eight parts at a time,
// their references and sums and values all on their way at once: the launch
// is a chain of latencies (Cut, parts, join of the groups), not of bytes.
template <class T, class C, bool PRE = false>
__global__ void __launch_bounds__(512) attend_join_kernel(const AttendArgs a) {
    constexpr int D = C::D, NG = 512 / D, U = 8;
    const int groups = blockDim.x / D;
    __shared__ float4 sum[NG][D];
    __shared__ float top[NG][4], total[NG][4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Cut cut = *cut_of(a, blockIdx.x);
    if (!cut.on) return;
    const int64_t c0 = blockIdx.x;
    const int n = (int)(cut.last - c0) + 1, q = blockIdx.y * 4;
    const int hk = cut.hc / a.groups, cg = cut.hc % a.groups;
    if (cg * C::kCols + q >= a.cols) return;
    const int grp = threadIdx.x / D, c = threadIdx.x % D / (D / 4), d = threadIdx.x % (D / 4) * 4;
    float m = kNone, l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp; i0 < n; i0 += groups * U) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + k * groups;
            ml[k] = make_float2(kNone, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const float* p = part_of<C>(a, c0 + i, i == 0 ? cut.which : 0);
                ml[k] = *reinterpret_cast<const float2*>(p + C::kCols * D + (q + c) * 2);
                v[k] = *reinterpret_cast<const float4*>(p + (q + c) * D + d);
            }
        }
        float to = m;
#pragma unroll
        for (int k = 0; k < U; ++k) to = fmaxf(to, ml[k].x);
        const float keep = exp2a(m - to);
        m = to;
        l *= keep;
        y = make_float4(y.x * keep, y.y * keep, y.z * keep, y.w * keep);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float f = exp2a(ml[k].x - m);
            l += ml[k].y * f;
            y.x += v[k].x * f;
            y.y += v[k].y * f;
            y.z += v[k].z * f;
            y.w += v[k].w * f;
        }
    }
    sum[grp][threadIdx.x % D] = y;
    if (d == 0) {
        top[grp][c] = m;
        total[grp][c] = l;
    }
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    const int oc = threadIdx.x / (D / 8), od = threadIdx.x % (D / 8);
    const Col col = column(a, hk, cg, q + oc, C::kCols);
    if (!col.on) return;
    float mx = kNone, ls = 0.f, r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < groups; ++k) mx = fmaxf(mx, top[k][oc]);
    for (int k = 0; k < groups; ++k) {
        const float f = exp2a(top[k][oc] - mx);
        ls += total[k][oc] * f;
        add8(r, &sum[k][oc * (D / 4) + 2 * od], f);
    }
    finish8<T, PRE>(a, cut.b, col, od * 8, r, ls, mx);
}

template <class C, bool PRE = false>
AttendEntry attend_entry(int dt, int most = INT32_MAX) {
    AttendEntry e;
    e.dt = dt;
    e.D = C::D;
    e.NT = C::NT;
    e.tok = C::kTok;
    e.per_sm = C::M;
    e.most = most;
    e.threads = C::W * 32;
    e.smem = C::kSmem;
    e.part = C::kCols * (C::D + 2);
    e.fn = dt == 1 ? (const void*)&attend_kernel<BF16, C, PRE>
                   : (const void*)&attend_kernel<F16, C, PRE>;
    e.join = dt == 1 ? (const void*)&attend_join_kernel<BF16, C, PRE>
                     : (const void*)&attend_join_kernel<F16, C, PRE>;
    return e;
}

}  // namespace rmsattn
