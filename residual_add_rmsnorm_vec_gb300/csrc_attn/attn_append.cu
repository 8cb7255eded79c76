// Append of new keys and values to the paged E4M3 cache.
//
// The unit of work is one block of 16 tokens of one sequence, one head, and
// k or v: its scale must be known before any of its codes.  Blocks that the
// new tokens of sequence b touch are numbered from (cu[b] >> 4) + 2 b: a
// sequence of n new tokens touches at most floor(n / 16) + 2 of them, and
// that sum grows by at least as much from b to b + 1, so the grid's size
// follows from the host's token and sequence counts alone and each unit
// finds its sequence by a search in cu.
#include "attn_common.cuh"

namespace rmsattn {

// Which block of which sequence unit u stands for.
struct Unit {
    int64_t b;       // sequence, or -1: none
    int64_t lo;      // position of the block's first token
    int64_t r0, r1;  // rows of the block that get new tokens: [r0, r1)
    int64_t src;     // row of k / v that goes to row r0
};

__device__ __forceinline__ Unit unit_of(const AppendArgs& a, int64_t u) {
    Unit w;
    w.b = -1;
    int64_t b, c0, c1, base;
    if (!a.cu) {
        b = u;
        c0 = u;
        c1 = u + 1;
        base = u;
        if (b >= a.B) return w;
    } else {
        // the last sequence whose base is at most u
        int64_t lo = 0, hi = a.B;  // base(lo) <= u < base(hi)
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (((int64_t)a.cu[mid] >> 4) + 2 * mid <= u) lo = mid;
            else hi = mid;
        }
        b = lo;
        c0 = a.cu[b];
        c1 = a.cu[b + 1];
        base = (c0 >> 4) + 2 * b;
    }
    const int64_t len = a.lengths[b];
    if (len < 0 || c0 < 0 || c1 <= c0 || c1 > a.T) return w;
    const int64_t n = c1 - c0;
    const int64_t blk = (len >> 4) + (u - base);
    if (blk < 0 || blk * kBlock >= len + n) return w;
    w.b = b;
    w.lo = blk * kBlock;
    w.r0 = len > w.lo ? len - w.lo : 0;
    w.r1 = len + n - w.lo < kBlock ? len + n - w.lo : kBlock;
    w.src = c0 + w.lo + w.r0 - len;
    return w;
}

// Scale of a block: a is its new elements' largest magnitude (fmaxf leaves NaN
// out; an infinity counts as the largest finite value).
__device__ __forceinline__ float next_scale(float before, float a) {
    float s = fmaxf(before, __fdiv_rn(fminf(a, 3.402823466e38f), 448.f));
    if ((a > 0.f || s > 0.f) && s < 1.17549435e-38f) s = 1.17549435e-38f;  // 1 / s stays finite
    return s;
}

// One block of 128 threads per unit, head and side, element by element.
template <class T>
__global__ void __launch_bounds__(128) append_simple(const AppendArgs a) {
    __shared__ float part[4];
    rmsn::pdl_launch_dependents(a.pdl);
    rmsn::pdl_wait(a.pdl);
    const Unit w = unit_of(a, blockIdx.x);
    if (w.b < 0) return;
    const int h = (int)blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const int64_t pg = page_of(a.c, a.table + w.b * a.table_stride, a.table_width, w.lo);
    if (pg < 0) {
        if (threadIdx.x == 0) atomicOr(a.status, kBadPage);
        return;
    }
    const int D = a.c.D;
    const int64_t in_page = w.lo % a.c.page;
    uint8_t* codes = (is_v ? a.c.v : a.c.k) + pg * a.c.page_stride +
                     ((int64_t)h * a.c.page + in_page) * D;
    float* scale = (is_v ? a.c.vs : a.c.ks) + pg * a.c.scale_stride +
                   (int64_t)h * (a.c.page / kBlock) + in_page / kBlock;
    const void* x = is_v ? a.v : a.k;
    const int64_t xs = is_v ? a.v_stride : a.k_stride;
    const int n = (int)(w.r1 - w.r0) * D;
    float m = 0.f;
    for (int e = threadIdx.x; e < n; e += 128)
        m = fmaxf(m, fabsf(load1<T>(x, (w.src + e / D) * xs + (int64_t)h * D + e % D)));
    m = rmsn::warp_max(m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    const float before = w.r0 > 0 ? *scale : 0.f;
    __syncthreads();
    const float s = next_scale(before, fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    if (threadIdx.x == 0) *scale = s;
    if (s > before) {
        const float ratio = before * r;
        for (int e = threadIdx.x; e < (int)w.r0 * D; e += 128)
            codes[e] = (uint8_t)pack_e4m3x2(rmsn::e4m3_value(codes[e]) * ratio, 0.f);
    }
    for (int e = threadIdx.x; e < n; e += 128) {
        const float v = load1<T>(x, (w.src + e / D) * xs + (int64_t)h * D + e % D);
        codes[w.r0 * D + e] = (uint8_t)pack_e4m3x2(v * r, 0.f);
    }
}

const void* append_simple_kernel(int dt) {
    return dt == 0 ? (const void*)&append_simple<F32>
                   : (dt == 1 ? (const void*)&append_simple<BF16> : (const void*)&append_simple<F16>);
}

}  // namespace rmsattn
