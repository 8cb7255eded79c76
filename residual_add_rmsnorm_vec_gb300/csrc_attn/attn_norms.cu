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
//
// Measured: 16384 x 8192 bf16 157 us, 6.84 TB/s (1.01 of the copy peak), with a gate for each
// token 225, 5.96 TB/s, for each sequence 162, over an fp32 stream 233, 6.9 TB/s; fp32 8192 x
// 8192 168, 6.4 TB/s.  4096 x 5120 bf16 to E4M3 with a gate for each sequence 31.5 us, 4.7 TB/s
// (26 without the gate): the rows' loads are what its warps wait for first, at 27 warps an SM
// (0.42), then the three row sums; issue slots are busy for 54 %.  8 x 4096 3.2 us (a launch,
// two loads and two sums).  Off the vectors' grid 4099 x 2045 31 us, 3.8 TB/s, 4096 x 8190 85 us,
// 3.2 TB/s (a weight is put together from two vectors; in fp32 from elements: 8192 x 8191 244).
// Rows above 16384 elements, and tensors whose rows' first elements do not lie on the grid, go
// element by element and meet memory again for each sum: 4096 x 20480 bf16 384 us (a floor of
// 99), 16384 x 8192 that begin one element off 723.
#include "attn_common.cuh"

namespace rmsattn {

namespace {

// V consecutive elements of T as they lie in memory.
template <class T, int V>
struct Raw {
    uint32_t u[V * T::kBytes >= 4 ? V * T::kBytes / 4 : 1];
};
template <class T, bool STREAM>
__device__ __forceinline__ Raw<T, 8> load(const void* p, int64_t e) {
    Raw<T, 8> v;
    if constexpr (T::kBytes == 4) {
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
    if (whole) return load<T, STREAM>(p, e);
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

// Eight elements as four pairs: two lanes an instruction.
template <class T>
__device__ __forceinline__ void pairs(const Raw<T, 8>& v, rmsn::F2 (&y)[4]) {
    float e[8];
    widen<T, 8>(v, e);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = rmsn::f2(e[2 * k], e[2 * k + 1]);
}
__device__ __forceinline__ void split(const rmsn::F2 (&y)[4], float (&e)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) rmsn::f2split(y[k], e[2 * k], e[2 * k + 1]);
}
__device__ __forceinline__ float squares(const float (&e)[8]) {
    const rmsn::F2 first = rmsn::f2(e[0], e[1]);
    rmsn::F2 s = rmsn::mul2(first, first);
#pragma unroll
    for (int k = 1; k < 4; ++k) {
        const rmsn::F2 y = rmsn::f2(e[2 * k], e[2 * k + 1]);
        s = rmsn::fma2(y, y, s);
    }
    float a, b;
    rmsn::f2split(s, a, b);
    return a + b;
}

// Elements j to j + 7 of a row of H that begins anywhere; those outside of it are zero.
// 16-bit ones come from the one or two vectors of memory that hold them, unless one of
// those lies in the row in part.  By elements alone 4099 x 2045 took 1.3 times as long.
template <class T>
__device__ __forceinline__ Raw<T, 8> load_any(const void* row, int j, int H) {
    if constexpr (T::kBytes == 2) {
        const uint16_t* q = static_cast<const uint16_t*>(row);
        const int d = (int)(reinterpret_cast<uintptr_t>(q + j) & 15) / 2;  // the same for all of the block
        const int e = j - d;
        auto in = [H](int e) { return e >= 0 && e + 8 <= H; };
        auto out = [H](int e) { return e + 8 <= 0 || e >= H; };
        if ((in(e) || out(e)) && (d == 0 || in(e + 8) || out(e + 8))) {
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            if (in(e)) lo = rmsn::ld_keep16(q + e);
            Raw<T, 8> v;
            if (d == 0) {
                v.u[0] = lo.x;
                v.u[1] = lo.y;
                v.u[2] = lo.z;
                v.u[3] = lo.w;
                return v;
            }
            if (in(e + 8)) hi = rmsn::ld_keep16(q + e + 8);
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t a[6], b[5];
#pragma unroll
            for (int k = 0; k < 6; ++k) a[k] = d & 4 ? w[k + 2] : w[k];
#pragma unroll
            for (int k = 0; k < 5; ++k) b[k] = d & 2 ? a[k + 1] : a[k];
#pragma unroll
            for (int k = 0; k < 4; ++k) v.u[k] = __byte_perm(b[k], b[k + 1], d & 1 ? 0x5432 : 0x3210);
            return v;
        }
    }
    return load_row<T, false>(row, j, j, H, false);
}

// The gate's row for row t (NULL: no gate), or false: the row belongs to no
// sequence and is left out.
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

// A row that is left out: zeros where the outputs are new, else as it was.
template <class T, class R, bool FP8>
__device__ __forceinline__ void leave_out(const NormsArgs& a, int64_t t) {
    const int64_t base = t * a.H;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        if (a.zero_out) {
            if constexpr (FP8) static_cast<uint8_t*>(a.out)[base + j] = 0;
            else store1<T>(a.out, base + j, 0.f);
        }
        if (a.zero_residual) store1<R>(a.residual_out, base + j, 0.f);
    }
    if (FP8 && a.zero_scale && threadIdx.x == 0) a.out_scale[t] = 0.f;
}

// 448 / top of an E4M3 row lies outside fp32's range for a row of less than 448 2^-128: y is
// lifted by 2^64 first there (an exact product; rows of weights or residuals near zero).
constexpr float kSmallRow = 0x1p-116f, kRowLift = 0x1p64f;

// y = (w + off) (h inv), in that order of roundings.
template <class T>
__device__ __forceinline__ void norm(const Raw<T, 8>& w, float off, float inv, const rmsn::F2 (&h)[4], rmsn::F2 (&y)[4]) {
    rmsn::F2 wv[4];
    pairs<T>(w, wv);
    const rmsn::F2 inv2 = rmsn::f2(inv, inv), off2 = rmsn::f2(off, off);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = rmsn::mul2(rmsn::mul2(h[k], inv2), rmsn::add2(wv[k], off2));
}
template <class T>
__device__ __forceinline__ Raw<T, 8> ones() {
    Raw<T, 8> v;
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
// bytes in each of them; the first and the last of a row go by elements.  Weights and
// gates begin anywhere.
template <class T, class R, int CH, bool FP8, bool RAGGED>
__global__ void __launch_bounds__(512, 2) norms_kernel(const NormsArgs a) {
    constexpr int V = 8;
    __shared__ float slot[3][32];
    rmsn::pdl_wait(a.pdl);
    rmsn::pdl_launch_dependents(a.pdl);
    const int64_t t = blockIdx.x, base = t * a.H;
    int64_t g0;
    if (!gate_row(a, t, &g0)) {
        leave_out<T, R, FP8>(a, t);
        return;
    }
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
    auto from = [&](const void* row, int c) {
        if constexpr (!RAGGED) return load<T, false>(row, j[c]);
        else return on[c] ? load_any<T>(row, j[c], a.H) : Raw<T, V>{};
    };
    auto weight = [&](const void* w, int c) { return w ? from(w, c) : ones<T>(); };
    const char* gate = a.gate ? static_cast<const char*>(a.gate) + g0 * T::kBytes : nullptr;
    // what lies outside of the row counts as zero
    auto clear = [&](int c, float (&v)[V]) {
        if (!RAGGED || whole[c]) return;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (!on[c] || j[c] + k < 0 || j[c] + k >= a.H) v[k] = 0.f;
    };
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float e[V];
        widen<T, V>(x[c], e);
        const float s = squares(e);
        sum += on[c] ? s : 0.f;  // (ragged rows' ends were loaded as zeros)
    }
    const float inv = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[0]), a.H, a.eps);
    const float post_off = a.post_w ? a.w_off : 0.f, off = a.w ? a.w_off : 0.f;
    const rmsn::F2 alpha = rmsn::f2(a.alpha, a.alpha);
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        rmsn::F2 v[4], p[4], h[4];
        pairs<T>(x[c], v);
        norm<T>(weight(a.post_w, c), post_off, inv, v, p);
        if (gate) {
            rmsn::F2 g[4];
            pairs<T>(from(gate, c), g);
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = rmsn::mul2(g[k], p[k]);
        }
        pairs<R>(r[c], h);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = rmsn::fma2(alpha, h[k], p[k]);
        float e[V];
        split(h, e);
        clear(c, e);
        r[c] = round_to<R, V>(e);
        if (on[c]) store_row<R>(a.residual_out, base + j[c], j[c], a.H, whole[c], r[c]);
        widen<R, V>(r[c], e);
        const float s = squares(e);
        sum += on[c] ? s : 0.f;
    }
    const float inv2 = rmsn::inv_rms(rmsn::block_allreduce<false>(sum, slot[1]), a.H, a.eps);
    if constexpr (!FP8) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            rmsn::F2 h[4], y[4];
            pairs<R>(r[c], h);
            norm<T>(weight(a.w, c), off, inv2, h, y);
            float e[V];
            split(y, e);
            if (on[c]) store_row<T>(a.out, base + j[c], j[c], a.H, whole[c], round_to<T, V>(e));
        }
    } else {  // y where x and h were, until the row's largest is known
        rmsn::F2 y[CH][4];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            rmsn::F2 h[4];
            pairs<R>(r[c], h);
            norm<T>(weight(a.w, c), off, inv2, h, y[c]);
            float e[V], m = 0.f;
            split(y[c], e);
            clear(c, e);
#pragma unroll
            for (int k = 0; k < V; ++k) m = fmaxf(m, fabsf(e[k]));
            top = fmaxf(top, on[c] ? m : 0.f);
        }
        top = rmsn::block_allreduce<true>(top, slot[2]);
        if (threadIdx.x == 0) a.out_scale[t] = __fdiv_rn(top, 448.f);
        if (top < kSmallRow) {
            top *= kRowLift;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k) y[c][k] = rmsn::mul2(y[c][k], rmsn::f2(kRowLift, kRowLift));
        }
        const float f = top > 0.f ? __fdiv_rn(448.f, top) : 0.f;
        const rmsn::F2 f2 = rmsn::f2(f, f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (!on[c]) continue;
            float e[V];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[c][k] = rmsn::mul2(y[c][k], f2);
            split(y[c], e);
            const uint32_t u[2] = {rmsn::pack_e4m3x4(e[0], e[1], e[2], e[3]), rmsn::pack_e4m3x4(e[4], e[5], e[6], e[7])};
            uint8_t* q = static_cast<uint8_t*>(a.out) + base + j[c];
            if (whole[c]) {
                rmsn::st_stream8(q, u);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (j[c] + k >= 0 && j[c] + k < a.H) q[k] = (uint8_t)(u[k / 4] >> k % 4 * 8);
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
    if (!gate_row(a, t, &g0)) {
        leave_out<T, R, FP8>(a, t);
        return;
    }
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
    float f = 1.f, lift = 1.f;
    if constexpr (FP8) {
        float top = 0.f;
        for (int j = threadIdx.x; j < a.H; j += blockDim.x) top = fmaxf(top, fabsf(out(j)));
        top = rmsn::block_allreduce<true>(top, slot[2]);
        if (threadIdx.x == 0) a.out_scale[t] = __fdiv_rn(top, 448.f);
        if (top < kSmallRow) lift = kRowLift;
        f = top > 0.f ? __fdiv_rn(448.f, top * lift) : 0.f;
    }
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
        const float y[1] = {out(j)};
        if constexpr (FP8) static_cast<uint8_t*>(a.out)[base + j] = (uint8_t)pack_e4m3x2(__fmul_rn(y[0] * lift, f), 0.f);
        else store<T, 1>(a.out, base + j, round_to<T, 1>(y));
    }
}

template <class T, class R, bool FP8, bool RAGGED>
const void* rows_kernel(int ch) {
    switch (ch) {
        case 1: return (const void*)&norms_kernel<T, R, 1, FP8, RAGGED>;
        case 2: return (const void*)&norms_kernel<T, R, 2, FP8, RAGGED>;
        case 3: return (const void*)&norms_kernel<T, R, 3, FP8, RAGGED>;
        default: return (const void*)&norms_kernel<T, R, 4, FP8, RAGGED>;
    }
}
template <class T, class R, bool FP8>
const void* kernel(bool ragged, int ch) {
    if (ch == 0) return (const void*)&norms_long_kernel<T, R, FP8>;
    return ragged ? rows_kernel<T, R, FP8, true>(ch) : rows_kernel<T, R, FP8, false>(ch);
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
