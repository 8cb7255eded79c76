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

// V consecutive elements of T as they lie in memory.
template <class T, int V>
struct Raw {
    uint32_t u[V * T::kBytes >= 4 ? V * T::kBytes / 4 : 1];
};
template <class T, int V, bool STREAM>
__device__ __forceinline__ Raw<T, V> load(const void* p, int64_t e) {
    Raw<T, V> v;
    if constexpr (V == 1) {
        if constexpr (T::kBytes == 4) v.u[0] = static_cast<const uint32_t*>(p)[e];
        else v.u[0] = static_cast<const uint16_t*>(p)[e];
    } else if constexpr (T::kBytes == 4) {
        static_assert(V == 8, "");
        const rmsn::V8 w = STREAM ? rmsn::ld_stream32(static_cast<const float*>(p) + e)
                                  : rmsn::ld_keep32(static_cast<const float*>(p) + e);
#pragma unroll
        for (int k = 0; k < 8; ++k) v.u[k] = w.u[k];
    } else {
        const uint16_t* q = static_cast<const uint16_t*>(p) + e;
        const uint4 w = STREAM ? rmsn::ld_stream16(q) : rmsn::ld_keep16(q);
        v.u[0] = w.x;
        v.u[1] = w.y;
        v.u[2] = w.z;
        v.u[3] = w.w;
    }
    return v;
}
template <class T, int V>
__device__ __forceinline__ void widen(const Raw<T, V>& v, float (&y)[V]) {
    if constexpr (T::kBytes == 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) y[k] = __uint_as_float(v.u[k]);
    } else if constexpr (V == 1) {
        y[0] = rmsn::lo2<T>(v.u[0]);
    } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            y[2 * k] = rmsn::lo2<T>(v.u[k]);
            y[2 * k + 1] = rmsn::hi2<T>(v.u[k]);
        }
    }
}
template <class T, int V>
__device__ __forceinline__ Raw<T, V> round_to(const float (&y)[V]) {
    Raw<T, V> v;
    if constexpr (T::kBytes == 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) v.u[k] = __float_as_uint(y[k]);
    } else if constexpr (V == 1) {
        v.u[0] = rmsn::pack2<T>(y[0], 0.f);
    } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) v.u[k] = rmsn::pack2<T>(y[2 * k], y[2 * k + 1]);
    }
    return v;
}
template <class T, int V>
__device__ __forceinline__ void store(void* p, int64_t e, const Raw<T, V>& v) {
    if constexpr (V == 1) {
        if constexpr (T::kBytes == 4) static_cast<uint32_t*>(p)[e] = v.u[0];
        else static_cast<uint16_t*>(p)[e] = (uint16_t)v.u[0];
    } else if constexpr (T::kBytes == 4) {
        rmsn::st_stream32(static_cast<float*>(p) + e, v.u);
    } else {
        rmsn::st_stream16(static_cast<uint16_t*>(p) + e, v.u);
    }
}

// The same at the ends of a row off the vectors' grid: of elements j to j + 7 those
// within [0, H).
template <class T, bool STREAM>
__device__ __forceinline__ Raw<T, 8> load_row(const void* p, int64_t e, int j, int H, bool whole) {
    if (whole) return load<T, 8, STREAM>(p, e);
    Raw<T, 8> v;
#pragma unroll
    for (uint32_t& u : v.u) u = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (j + k < 0 || j + k >= H) continue;
        if constexpr (T::kBytes == 4) v.u[k] = static_cast<const uint32_t*>(p)[e + k];
        else v.u[k / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[e + k] << (k & 1) * 16;
    }
    return v;
}
template <class T>
__device__ __forceinline__ void store_row(void* p, int64_t e, int j, int H, bool whole, const Raw<T, 8>& v) {
    if (whole) {
        store<T, 8>(p, e, v);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (j + k < 0 || j + k >= H) continue;
        if constexpr (T::kBytes == 4) static_cast<uint32_t*>(p)[e + k] = v.u[k];
        else static_cast<uint16_t*>(p)[e + k] = (uint16_t)(v.u[k / 2] >> (k & 1) * 16);
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

// y = (w + off) (h inv), in that order of roundings; w of ones (no weight) with off 0.
template <class T, int V>
__device__ __forceinline__ void norm(const Raw<T, V>& w, float off, float inv, const float (&h)[V], float (&y)[V]) {
    float wv[V];
    widen<T, V>(w, wv);
    if constexpr (V == 1) {
        y[0] = __fmul_rn(__fmul_rn(h[0], inv), __fadd_rn(wv[0], off));
    } else {  // two lanes an instruction, each rounded as above
        const rmsn::F2 inv2 = rmsn::f2(inv, inv), off2 = rmsn::f2(off, off);
#pragma unroll
        for (int k = 0; k < V; k += 2)
            rmsn::f2split(rmsn::mul2(rmsn::mul2(rmsn::f2(h[k], h[k + 1]), inv2),
                                     rmsn::add2(rmsn::f2(wv[k], wv[k + 1]), off2)),
                          y[k], y[k + 1]);
    }
}
template <class T, int V>
__device__ __forceinline__ Raw<T, V> ones() {
    Raw<T, V> v;
#pragma unroll
    for (uint32_t& u : v.u) u = rmsn::ones_word<T>();
    return v;
}

// A row held in registers: CH vectors of eight elements a thread.  The row's loads are
// issued at an address that is right for each (past the row's end: the row's begin),
// not behind a branch, where they would be waited for.  The weights and gates, from L1
// and L2, are loaded where they are used: 64 registers, 1024 threads an SM.
//
// RAGGED: rows off the vectors' grid.  All of a token's rows begin at the same element
// t H of their tensors, so that the vectors at multiples of eight of those lie on 16
// bytes in each of them; the first and the last of a row go by elements, and so do the
// weights, which are counted from the row's begin.
template <class T, class R, int CH, bool FP8, bool RAGGED>
__global__ void __launch_bounds__(512, 2) norms_kernel(const NormsArgs a) {
    constexpr int V = 8;
    __shared__ float slot[3][32];
    rmsn::pdl_wait(a.pdl);
    rmsn::pdl_launch_dependents(a.pdl);
    const int64_t t = blockIdx.x, base = t * a.H;
    int64_t g0;
    if (!gate_row(a, t, &g0)) return;
    const int shift = RAGGED ? (int)(base & 7) : 0;
    Raw<T, V> x[CH];
    Raw<R, V> r[CH];
    int j[CH];
    bool on[CH], whole[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        j[c] = (threadIdx.x + c * blockDim.x) * V - shift;
        on[c] = j[c] < a.H;
        whole[c] = !RAGGED || (j[c] >= 0 && j[c] + V <= a.H);
        if (!on[c]) {
            j[c] = 0;
            whole[c] = !RAGGED;
        }
        x[c] = load_row<T, true>(a.x, base + j[c], j[c], on[c] ? a.H : 0, whole[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) r[c] = load_row<R, true>(a.residual, base + j[c], j[c], on[c] ? a.H : 0, whole[c]);
    auto weight = [&](const void* w, int c) {
        if (!w) return ones<T, V>();
        return load_row<T, false>(w, j[c], j[c], on[c] ? a.H : 0, !RAGGED);
    };
    // a gate's row for each token lies as the token's other rows do
    const bool straight = !RAGGED || (((g0 - base) & 7) == 0 && (reinterpret_cast<uintptr_t>(a.gate) & (8 * T::kBytes - 1)) == 0);
    auto inside = [&](int c, int k) { return on[c] && (!RAGGED || (j[c] + k >= 0 && j[c] + k < a.H)); };
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float v[V];
        widen<T, V>(x[c], v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (!RAGGED) v[k] = on[c] ? v[k] : 0.f;  // (ragged: zeros already)
            sum = __fmaf_rn(v[k], v[k], sum);
        }
    }
    const float inv = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[0]), a.H, a.eps);
    const float post_off = a.post_w ? a.w_off : 0.f, off = a.w ? a.w_off : 0.f;
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float v[V], p[V], h[V];
        widen<T, V>(x[c], v);
        norm<T, V>(weight(a.post_w, c), post_off, inv, v, p);
        if (a.gate) {
            float g[V];
            widen<T, V>(load_row<T, false>(a.gate, g0 + j[c], j[c], on[c] ? a.H : 0, whole[c] && straight), g);
#pragma unroll
            for (int k = 0; k < V; ++k) p[k] = __fmul_rn(g[k], p[k]);
        }
        widen<R, V>(r[c], h);
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = __fmaf_rn(a.alpha, h[k], p[k]);
        r[c] = round_to<R, V>(h);
        if (on[c]) store_row<R>(a.residual_out, base + j[c], j[c], a.H, whole[c], r[c]);
        widen<R, V>(r[c], h);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            h[k] = inside(c, k) ? h[k] : 0.f;
            sum = __fmaf_rn(h[k], h[k], sum);
        }
    }
    const float inv2 = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[1]), a.H, a.eps);
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float h[V], y[V];
        widen<R, V>(r[c], h);
        norm<T, V>(weight(a.w, c), off, inv2, h, y);
        if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < V; ++k) top = fmaxf(top, inside(c, k) ? fabsf(y[k]) : 0.f);
        } else {
            if (on[c]) store_row<T>(a.out, base + j[c], j[c], a.H, whole[c], round_to<T, V>(y));
        }
    }
    if constexpr (FP8) {
        top = rmsn::block_allreduce<true>(top, slot[2]);
        const float f = top > 0.f ? __fdiv_rn(448.f, top) : 0.f;
        if (threadIdx.x == 0) a.out_scale[t] = __fdiv_rn(top, 448.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float h[V], y[V];
            widen<R, V>(r[c], h);
            norm<T, V>(weight(a.w, c), off, inv2, h, y);
            if (!on[c]) continue;
            if (whole[c]) {
                store_codes<V>(a.out, base + j[c], y, f);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float one[1] = {y[k]};
                    if (inside(c, k)) store_codes<1>(a.out, base + j[c] + k, one, f);
                }
            }
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
    auto weight = [](const void* w, int64_t e, float off) { return w ? __fadd_rn(load1<T>(w, e), off) : 1.f; };
    float sum = 0.f;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        const float x = load1<T>(a.x, base + j);
        sum = __fmaf_rn(x, x, sum);
    }
    const float inv = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[0]), a.H, a.eps);
    sum = 0.f;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        float p = __fmul_rn(__fmul_rn(load1<T>(a.x, base + j), inv), weight(a.post_w, j, a.w_off));
        if (a.gate) p = __fmul_rn(load1<T>(a.gate, g0 + j), p);
        float h[1] = {__fmaf_rn(a.alpha, load1<R>(a.residual, base + j), p)};
        const Raw<R, 1> kept = round_to<R, 1>(h);
        store<R, 1>(a.residual_out, base + j, kept);
        widen<R, 1>(kept, h);
        sum = __fmaf_rn(h[0], h[0], sum);
    }
    const float inv2 = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[1]), a.H, a.eps);
    auto out = [&](int j) {
        return __fmul_rn(__fmul_rn(load1<R>(a.residual_out, base + j), inv2), weight(a.w, j, a.w_off));
    };
    float f = 1.f;
    if constexpr (FP8) {
        float top = 0.f;
        for (int j = threadIdx.x; j < a.H; j += blockDim.x) top = fmaxf(top, fabsf(out(j)));
        top = rmsn::block_allreduce<true>(top, slot[2]);
        f = top > 0.f ? __fdiv_rn(448.f, top) : 0.f;
        if (threadIdx.x == 0) a.out_scale[t] = __fdiv_rn(top, 448.f);
    }
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        const float y[1] = {out(j)};
        if constexpr (FP8) store_codes<1>(a.out, base + j, y, f);
        else store<T, 1>(a.out, base + j, round_to<T, 1>(y));
    }
}

template <class T, class R, bool FP8>
const void* kernel(bool ragged, int ch) {
    if (ch == 0) return (const void*)&norms_long_kernel<T, R, FP8>;
    if (ragged)
        return ch == 1 ? (const void*)&norms_kernel<T, R, 1, FP8, true>
                       : (ch == 2 ? (const void*)&norms_kernel<T, R, 2, FP8, true>
                                  : (const void*)&norms_kernel<T, R, 4, FP8, true>);
    return ch == 1 ? (const void*)&norms_kernel<T, R, 1, FP8, false>
                   : (ch == 2 ? (const void*)&norms_kernel<T, R, 2, FP8, false>
                              : (const void*)&norms_kernel<T, R, 4, FP8, false>);
}

}  // namespace

const void* norms_kernel_of(int dt, bool r32, bool fp8, bool ragged, int ch) {
    if (dt == 0) return fp8 ? kernel<F32, F32, true>(ragged, ch) : kernel<F32, F32, false>(ragged, ch);
    if (dt == 1) {
        if (r32) return fp8 ? kernel<BF16, F32, true>(ragged, ch) : kernel<BF16, F32, false>(ragged, ch);
        return fp8 ? kernel<BF16, BF16, true>(ragged, ch) : kernel<BF16, BF16, false>(ragged, ch);
    }
    if (r32) return fp8 ? kernel<F16, F32, true>(ragged, ch) : kernel<F16, F32, false>(ragged, ch);
    return fp8 ? kernel<F16, F16, true>(ragged, ch) : kernel<F16, F16, false>(ragged, ch);
}

}  // namespace rmsattn
