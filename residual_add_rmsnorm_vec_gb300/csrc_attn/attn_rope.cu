// QK norm and rotary positions with several axes.
//
// A pair (a, b) of a head is turned by the angle 2 pi frac(pos * f), f in
// turns per position.  f is held as a 64-bit fraction of one turn, so the
// 64-bit product with an integer position, taken modulo 2^64, IS the phase
// modulo one turn: two integer multiply-adds replace an fp64 product and a
// range reduction, and far positions lose nothing.  The top 32 bits, as a
// signed number, are the phase in (-1/2, 1/2] turns = (-1, 1] half turns for
// sincospi, which is accurate to an ulp or two of fp32.
#include "attn_common.cuh"

namespace rmsattn {

__device__ __forceinline__ int64_t position(const RopeArgs& a, int p, int64_t t) {
    uint32_t ax = (uint32_t)a.axis[p];
    if (ax >= (uint32_t)a.n_axes) ax = 0;  // a table for more axes than positions
    const int64_t e = (int64_t)ax * a.pos_stride + t;
    return a.pos64 ? static_cast<const int64_t*>(a.pos)[e]
                   : (int64_t) static_cast<const int32_t*>(a.pos)[e];
}

// cos and sin of pair p's angle at token t.
__device__ __forceinline__ float2 turn(const RopeArgs& a, int p, int64_t t) {
    const uint64_t phase = a.turns[p] * (uint64_t)position(a, p, t);
    float2 cs;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
    return cs;
}

// Any head size, stride and alignment: one warp per head, element by element.
// Each lane writes only the pairs that it has read itself, after the whole
// head has been read for its norm, so the output may be the input.
template <class T>
__global__ void __launch_bounds__(256) rope_generic(const RopeArgs a) {
    rmsn::pdl_launch_dependents(a.pdl);
    rmsn::pdl_wait(a.pdl);
    const int lane = threadIdx.x & 31;
    const int64_t heads = a.Hq + a.Hk, total = a.T * heads;
    const int P = a.R / 2;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < total;
         u += (int64_t)gridDim.x * 8) {
        const int64_t t = u / heads;
        const int h = (int)(u % heads);
        const bool is_q = h < a.Hq;
        const void* x = is_q ? a.q : a.k;
        void* o = is_q ? a.qo : a.ko;
        const void* w = is_q ? a.qw : a.kw;
        const int64_t hd = (int64_t)(is_q ? h : h - a.Hq) * a.D;
        const int64_t xe = t * (is_q ? a.qs : a.ks) + hd, oe = t * (is_q ? a.qos : a.kos) + hd;
        float inv = 1.f;
        if (a.norm) {
            float acc = 0.f;
            for (int e = lane; e < a.D; e += 32) {
                const float v = load1<T>(x, xe + e);
                acc = fmaf(v, v, acc);
            }
            acc = rmsn::warp_sum(acc);
            inv = __frsqrt_rn(__fadd_rn(__fdiv_rn(acc, (float)a.D), a.eps));
        }
        auto y = [&](int e) {
            const float v = load1<T>(x, xe + e);
            if (!a.norm) return v;
            const float wv = w ? load1<T>(w, e) : 1.f;
            return (wv + a.woff) * (v * inv);
        };
        for (int p = lane; p < P; p += 32) {
            const int i = a.interleaved ? 2 * p : p, j = a.interleaved ? 2 * p + 1 : p + P;
            const float2 cs = turn(a, p, t);
            const float yi = y(i), yj = y(j);
            store1<T>(o, oe + i, yi * cs.x - yj * cs.y);
            store1<T>(o, oe + j, yj * cs.x + yi * cs.y);
        }
        for (int e = a.R + lane; e < a.D; e += 32) store1<T>(o, oe + e, y(e));
    }
}

const void* rope_generic_kernel(int dt) {
    return dt == 0 ? (const void*)&rope_generic<F32>
                   : (dt == 1 ? (const void*)&rope_generic<BF16> : (const void*)&rope_generic<F16>);
}

}  // namespace rmsattn
