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
    int r0, r1;      // rows of the block that get new tokens: [r0, r1)
    int64_t src;     // row of k / v that would go to row 0
};

// The warp's lanes search together, 32 sequences a step.
__device__ __forceinline__ Unit unit_of(const AppendArgs& a, int64_t u) {
    Unit w;
    w.b = -1;
    int64_t b, c0, c1, base;
    if (!a.cu) {
        b = u;
        c0 = u;
        c1 = u + 1;
        base = u;
    } else {
        // the last sequence whose base is at most u
        int64_t lo = 0, n = a.B;
        while (n > 1) {
            const int64_t step = (n + 31) / 32, i = (threadIdx.x & 31) * step;
            const bool in = i < n && ((int64_t)a.cu[lo + i] >> 4) + 2 * (lo + i) <= u;
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, in) | 1u;
            const int64_t k = 31 - __clz(hit);
            lo += k * step;
            n = n - k * step < step ? n - k * step : step;
        }
        b = lo;
        c0 = a.cu[b];
        c1 = a.cu[b + 1];
        base = (c0 >> 4) + 2 * b;
    }
    const int64_t len = a.lengths[b];
    if (len < 0 || c0 < 0 || c1 <= c0 || c1 > a.T || u < base) return w;
    const int64_t n = c1 - c0;
    const int64_t blk = (len >> 4) + (u - base);
    if (blk * kBlock >= len + n) return w;
    w.b = b;
    w.lo = blk * kBlock;
    w.r0 = len > w.lo ? (int)(len - w.lo) : 0;
    w.r1 = len + n - w.lo < kBlock ? (int)(len + n - w.lo) : kBlock;
    w.src = c0 + w.lo - len;
    return w;
}

// Scale of a block: a is its new elements' largest magnitude (fmaxf leaves NaN
// out; an infinity counts as the largest finite value).
__device__ __forceinline__ float next_scale(float before, float a) {
    float s = fmaxf(before, __fdiv_rn(fminf(a, 3.402823466e38f), 448.f));
    if ((a > 0.f || s > 0.f) && s < 1.17549435e-38f) s = 1.17549435e-38f;  // 1 / s stays finite
    return s;
}

// One warp per unit, head and side.  D / 8 lanes hold a token, eight elements
// each, 32 / (D / 8) tokens at a time, so the whole block of 16 tokens is read
// in one go (4 KB in bf16 at head_dim 128: enough bytes in flight without a
// ring), stays in registers while the warp finds its largest magnitude, and is
// written once.  VEC: 16-byte loads; else element by element.
// Bound by DRAM: 32000 tokens x 8 heads x 128 bf16 (197 MB read and written)
// in 32.6 us on a GB300, 0.89 of the copy peak; a block of 128 threads that
// read its 16 tokens twice, element by element, took 185 us, and this kernel
// with its values widened while held (100 registers, 16 warps an SM) 43.
// One token to each of 64 sequences: 3.8 us, four dependent reads (length,
// page, scale, codes) and the launch.
// Held as loaded: the values are widened twice (for the maximum in the 16-bit
// type itself), so that 64 registers do and 32 warps share an SM.
template <class T, int D>
struct AppendBounds {
    static constexpr int kHeld = D / 16 * T::kBytes * 2;  // registers of a lane's elements
    static constexpr int kBlocks = kHeld <= 32 ? 4 : (kHeld <= 64 ? 2 : 1);
};
// Largest magnitude of the 16-bit pairs a and b, lane by lane (the sign bits
// of the result say nothing); NaN is left out.
template <class T>
__device__ __forceinline__ uint32_t absmax16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (rmsn::IsF16<T>::value) asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <class T, int D, bool VEC>
__global__ void __launch_bounds__(256, AppendBounds<T, D>::kBlocks) append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 8, RPS = 32 / LPR, N = kBlock / RPS;
    constexpr int NW = T::kBytes * 2;  // words of eight elements
    rmsn::pdl_launch_dependents(a.pdl);
    rmsn::pdl_wait(a.pdl);
    const int hs = (int)blockIdx.y * (int)(blockDim.x >> 5) + (int)(threadIdx.x >> 5);
    if (hs >= 2 * a.c.H) return;
    const Unit w = unit_of(a, blockIdx.x);
    if (w.b < 0) return;
    const int h = hs >> 1, lane = threadIdx.x & 31, r = lane / LPR, d = lane % LPR * 8;
    const bool is_v = hs & 1;
    const void* x = is_v ? a.v : a.k;
    const int64_t xs = is_v ? a.v_stride : a.k_stride;
    uint32_t u[N][NW];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = i * RPS + r;
#pragma unroll
        for (int k = 0; k < NW; ++k) u[i][k] = 0;
        if (row < w.r0 || row >= w.r1) continue;
        const int64_t e = (w.src + row) * xs + (int64_t)h * D + d;
        if constexpr (VEC) {
            const char* p = static_cast<const char*>(x) + e * T::kBytes;
#pragma unroll
            for (int k = 0; k < NW; k += 4) {
                const uint4 v = rmsn::ld_stream16(p + 4 * k);
                u[i][k] = v.x;
                u[i][k + 1] = v.y;
                u[i][k + 2] = v.z;
                u[i][k + 3] = v.w;
            }
        } else if constexpr (T::kBytes == 4) {
#pragma unroll
            for (int k = 0; k < 8; ++k) u[i][k] = static_cast<const uint32_t*>(x)[e + k];
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(x) + e;
#pragma unroll
            for (int k = 0; k < 4; ++k) u[i][k] = (uint32_t)p[2 * k] | ((uint32_t)p[2 * k + 1] << 16);
        }
    }
    const int64_t pg = page_of(a.c, a.table + w.b * a.table_stride, a.table_width, w.lo);
    if (pg < 0) {
        if (lane == 0) atomicOr(a.status, kBadPage);
        return;
    }
    const int in_page = (int)(w.lo % a.c.page);
    uint8_t* codes = (is_v ? a.c.v : a.c.k) + pg * a.c.page_stride +
                     ((int64_t)h * a.c.page + in_page) * D + d;
    float* scale = (is_v ? a.c.vs : a.c.ks) + pg * a.c.scale_stride +
                   (int64_t)h * (a.c.page / kBlock) + in_page / kBlock;
    const float before = w.r0 > 0 ? *scale : 0.f;
    auto value = [&](int i, int k) {  // element k of row i
        if constexpr (T::kBytes == 4) return __uint_as_float(u[i][k]);
        else return (k & 1) ? rmsn::hi2<T>(u[i][k >> 1]) : rmsn::lo2<T>(u[i][k >> 1]);
    };
    float m = 0.f;
    if constexpr (T::kBytes == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < 8; k += 2) m = rmsn::absmax3(m, value(i, k), value(i, k + 1));
    } else {
        uint32_t m2 = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < NW; ++k) m2 = absmax16x2<T>(m2, u[i][k]);
        m = rmsn::absmax3(0.f, rmsn::lo2<T>(m2), rmsn::hi2<T>(m2));
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < NW; ++k) asm volatile("" : "+r"(u[i][k]));
    }
    m = rmsn::warp_max(m);
    const float s = next_scale(before, m);
    const float f = s > 0.f ? __frcp_rn(s) : 0.f;
    __syncwarp();  // every lane has read the scale before
    if (lane == 0) *scale = s;
    if (s > before && w.r0 > 0) {  // the older codes follow the scale
        const float ratio = before * f;
#pragma unroll 4
        for (int i = 0; i < N; ++i) {
            const int row = i * RPS + r;
            if (row >= w.r0) continue;
            uint2 c = *reinterpret_cast<const uint2*>(codes + row * D);
            uint32_t out[2];
            const uint32_t in[2] = {c.x, c.y};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t lo = e4m3x2_to_f16x2(in[k]), hi = e4m3x2_to_f16x2(in[k] >> 16);
                out[k] = rmsn::pack_e4m3x4(rmsn::lo2<F16>(lo) * ratio, rmsn::hi2<F16>(lo) * ratio,
                                           rmsn::lo2<F16>(hi) * ratio, rmsn::hi2<F16>(hi) * ratio);
            }
            *reinterpret_cast<uint2*>(codes + row * D) = make_uint2(out[0], out[1]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = i * RPS + r;
        if (row < w.r0 || row >= w.r1) continue;
        uint32_t out[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
        {
            const rmsn::F2 f2 = rmsn::f2(f, f);
            float x[4];
            rmsn::f2split(rmsn::mul2(rmsn::f2(value(i, 4 * k), value(i, 4 * k + 1)), f2), x[0], x[1]);
            rmsn::f2split(rmsn::mul2(rmsn::f2(value(i, 4 * k + 2), value(i, 4 * k + 3)), f2), x[2], x[3]);
            out[k] = rmsn::pack_e4m3x4(x[0], x[1], x[2], x[3]);
        }
        *reinterpret_cast<uint2*>(codes + row * D) = make_uint2(out[0], out[1]);
    }
}

template <int D, bool VEC>
const void* append_of(int dt) {
    return dt == 0 ? (const void*)&append_kernel<F32, D, VEC>
                   : (dt == 1 ? (const void*)&append_kernel<BF16, D, VEC>
                              : (const void*)&append_kernel<F16, D, VEC>);
}

const void* append_kernel_of(int dt, int D, bool vec) {
    if (D == 64) return vec ? append_of<64, true>(dt) : append_of<64, false>(dt);
    if (D == 128) return vec ? append_of<128, true>(dt) : append_of<128, false>(dt);
    return vec ? append_of<256, true>(dt) : append_of<256, false>(dt);
}

}  // namespace rmsattn
