// The end of one block and the begin of the next, a row of H elements:
//
//   p = (post_w + w_off) x rsqrt(mean(x^2) + eps)
//   h = RN(residual_scale residual + gate p)            -> residual_out
//   y = (w + w_off) h rsqrt(mean(h^2) + eps)            -> out (x's type, or E4M3 codes and max|y| / 448)
//
// What bounds it: DRAM, 8 H bytes a row in 16 bits (10 with a gate for every
// token).  Two row sums stand in a row, one behind the other, so a row's loads
// are issued at once and held in registers (x, then h in its place), and the
// blocks of other rows on the SM stream while this one waits: a block per row,
// the block scheduler brings in the next as soon as one retires.
#include "attn_common.cuh"

namespace rmsattn {

namespace {

// V consecutive elements of T as floats, from element e on.
template <class T, int V, bool STREAM>
__device__ __forceinline__ void load(const void* p, int64_t e, float (&y)[V]) {
    if constexpr (V == 1) {
        y[0] = load1<T>(p, e);
    } else if constexpr (T::kBytes == 4) {
        static_assert(V == 8, "");
        const rmsn::V8 v = STREAM ? rmsn::ld_stream32(static_cast<const float*>(p) + e)
                                  : rmsn::ld_keep32(static_cast<const float*>(p) + e);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(v.u[k]);
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + e;
        const uint4 w = STREAM ? rmsn::ld_stream16(q) : rmsn::ld_keep16(q);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[2 * k] = rmsn::lo2<T>(u[k]);
            y[2 * k + 1] = rmsn::hi2<T>(u[k]);
        }
    }
}

// Rounds to T, stores, and leaves the rounded values in y.
template <class T, int V>
__device__ __forceinline__ void store_rounded(void* p, int64_t e, float (&y)[V]) {
    if constexpr (T::kBytes == 4) {
        if constexpr (V == 1) {
            static_cast<float*>(p)[e] = y[0];
        } else {
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(y[k]);
            rmsn::st_stream32(static_cast<float*>(p) + e, u);
        }
    } else if constexpr (V == 1) {
        const uint32_t u = rmsn::pack2<T>(y[0], 0.f);
        static_cast<uint16_t*>(p)[e] = (uint16_t)u;
        y[0] = rmsn::lo2<T>(u);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            u[k] = rmsn::pack2<T>(y[2 * k], y[2 * k + 1]);
            y[2 * k] = rmsn::lo2<T>(u[k]);
            y[2 * k + 1] = rmsn::hi2<T>(u[k]);
        }
        rmsn::st_stream16(static_cast<uint16_t*>(p) + e, u);
    }
}

template <int V>
__device__ __forceinline__ void store_codes(void* p, int64_t e, const float (&y)[V], float f) {
    uint8_t* q = static_cast<uint8_t*>(p) + e;
    if constexpr (V == 1) {
        *q = (uint8_t)pack_e4m3x2(__fmul_rn(y[0], f), 0.f);
    } else {
        uint32_t u[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            u[k] = rmsn::pack_e4m3x4(__fmul_rn(y[4 * k], f), __fmul_rn(y[4 * k + 1], f),
                                     __fmul_rn(y[4 * k + 2], f), __fmul_rn(y[4 * k + 3], f));
        rmsn::st_stream8(q, u);
    }
}

// The gate's row for row t (NULL: no gate), or false: the row belongs to no
// sequence and is left as it is.
__device__ __forceinline__ bool gate_row(const NormsArgs& a, int64_t t, int64_t* at) {
    *at = t * a.gate_stride;
    if (!a.index) return true;
    const int32_t i = a.index[t];
    if (i >= a.n_gates) {
        if (threadIdx.x == 0) atomicOr(a.status, kBadPage);
        return false;
    }
    *at = i * a.gate_stride;
    return i >= 0;
}

// y of a vector: from h and the weights.
template <class T, int V>
__device__ __forceinline__ void norm(const void* w, int64_t j, float off, float inv, const float (&h)[V],
                                     float (&y)[V]) {
    float wv[V];
    if (w) load<T, V, false>(w, j, wv);
#pragma unroll
    for (int k = 0; k < V; ++k) y[k] = __fmul_rn(__fmul_rn(h[k], inv), w ? __fadd_rn(wv[k], off) : 1.f);
}

// A row held in registers: CH vectors of V elements a thread.
template <class T, class R, int V, int CH, bool FP8>
__global__ void __launch_bounds__(CH * V >= 32 ? 512 : 1024) norms_kernel(const NormsArgs a) {
    __shared__ float slot[3][32];
    rmsn::pdl_wait(a.pdl);
    rmsn::pdl_launch_dependents(a.pdl);
    const int64_t t = blockIdx.x, base = t * a.H;
    const int step = blockDim.x * V;
    int64_t g0;
    if (!gate_row(a, t, &g0)) return;
    float x[CH][V], r[CH][V];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int j = threadIdx.x * V + c * step;
        if (j < a.H) load<T, V, true>(a.x, base + j, x[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int j = threadIdx.x * V + c * step;
        if (j < a.H) load<R, V, true>(a.residual, base + j, r[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (threadIdx.x * V + c * step < a.H) {
#pragma unroll
            for (int k = 0; k < V; ++k) sum = __fmaf_rn(x[c][k], x[c][k], sum);
        }
    const float inv = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[0]), a.H, a.eps);
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int j = threadIdx.x * V + c * step;
        if (j >= a.H) continue;
        float p[V], g[V];
        norm<T, V>(a.post_w, j, a.w_off, inv, x[c], p);
        if (a.gate) load<T, V, false>(a.gate, g0 + j, g);
#pragma unroll
        for (int k = 0; k < V; ++k)
            x[c][k] = __fmaf_rn(a.alpha, r[c][k], a.gate ? __fmul_rn(g[k], p[k]) : p[k]);
        store_rounded<R, V>(a.residual_out, base + j, x[c]);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = __fmaf_rn(x[c][k], x[c][k], sum);
    }
    const float inv2 = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[1]), a.H, a.eps);
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int j = threadIdx.x * V + c * step;
        if (j >= a.H) continue;
        norm<T, V>(a.w, j, a.w_off, inv2, x[c], x[c]);
        if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < V; ++k) top = fmaxf(top, fabsf(x[c][k]));
        } else {
            store_rounded<T, V>(a.out, base + j, x[c]);
        }
    }
    if constexpr (FP8) {
        top = rmsn::block_allreduce<true>(top, slot[2]);
        const float f = top > 0.f ? __fdiv_rn(448.f, top) : 0.f;
        if (threadIdx.x == 0) a.out_scale[t] = __fdiv_rn(top, 448.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = threadIdx.x * V + c * step;
            if (j < a.H) store_codes<V>(a.out, base + j, x[c], f);
        }
    }
}

// Rows of any length: h is read again from residual_out, by the thread that
// wrote it.
template <class T, class R, bool FP8>
__global__ void __launch_bounds__(1024) norms_long_kernel(const NormsArgs a) {
    __shared__ float slot[3][32];
    rmsn::pdl_wait(a.pdl);
    rmsn::pdl_launch_dependents(a.pdl);
    const int64_t t = blockIdx.x, base = t * a.H;
    int64_t g0;
    if (!gate_row(a, t, &g0)) return;
    float sum = 0.f, h[1], y[1], g[1];
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        load<T, 1, true>(a.x, base + j, h);
        sum = __fmaf_rn(h[0], h[0], sum);
    }
    const float inv = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[0]), a.H, a.eps);
    sum = 0.f;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        load<T, 1, true>(a.x, base + j, h);
        norm<T, 1>(a.post_w, j, a.w_off, inv, h, y);
        load<R, 1, true>(a.residual, base + j, h);
        if (a.gate) {
            load<T, 1, false>(a.gate, g0 + j, g);
            y[0] = __fmul_rn(g[0], y[0]);
        }
        h[0] = __fmaf_rn(a.alpha, h[0], y[0]);
        store_rounded<R, 1>(a.residual_out, base + j, h);
        sum = __fmaf_rn(h[0], h[0], sum);
    }
    const float inv2 = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[1]), a.H, a.eps);
    float f = 1.f;
    if constexpr (FP8) {
        float top = 0.f;
        for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
            h[0] = load1<R>(a.residual_out, base + j);
            norm<T, 1>(a.w, j, a.w_off, inv2, h, y);
            top = fmaxf(top, fabsf(y[0]));
        }
        top = rmsn::block_allreduce<true>(top, slot[2]);
        f = top > 0.f ? __fdiv_rn(448.f, top) : 0.f;
        if (threadIdx.x == 0) a.out_scale[t] = __fdiv_rn(top, 448.f);
    }
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        h[0] = load1<R>(a.residual_out, base + j);
        norm<T, 1>(a.w, j, a.w_off, inv2, h, y);
        if constexpr (FP8) store_codes<1>(a.out, base + j, y, f);
        else store_rounded<T, 1>(a.out, base + j, y);
    }
}

template <class T, class R, bool FP8>
const void* kernel(int v, int ch) {
    if (v == 1) return ch == 0 ? (const void*)&norms_long_kernel<T, R, FP8> : (const void*)&norms_kernel<T, R, 1, 8, FP8>;
    return ch == 1 ? (const void*)&norms_kernel<T, R, 8, 1, FP8>
                   : (ch == 2 ? (const void*)&norms_kernel<T, R, 8, 2, FP8>
                              : (const void*)&norms_kernel<T, R, 8, 4, FP8>);
}

}  // namespace

const void* norms_kernel_of(int dt, bool r32, bool fp8, int v, int ch) {
    if (dt == 0) return fp8 ? kernel<F32, F32, true>(v, ch) : kernel<F32, F32, false>(v, ch);
    if (dt == 1) {
        if (r32) return fp8 ? kernel<BF16, F32, true>(v, ch) : kernel<BF16, F32, false>(v, ch);
        return fp8 ? kernel<BF16, BF16, true>(v, ch) : kernel<BF16, BF16, false>(v, ch);
    }
    if (r32) return fp8 ? kernel<F16, F32, true>(v, ch) : kernel<F16, F32, false>(v, ch);
    return fp8 ? kernel<F16, F16, true>(v, ch) : kernel<F16, F16, false>(v, ch);
}

}  // namespace rmsattn
