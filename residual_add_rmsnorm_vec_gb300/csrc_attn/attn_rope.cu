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

// ---------------------------------------------------------------- 16-byte vectors
//
// A lane holds two 16-byte chunks of a head, chosen so that every pair lies
// within the lane: with halves (i, i + R / 2), chunk c of the first half and
// chunk c of the second; with neighbours (2p, 2p + 1) any two chunks will do,
// so the same two are taken; beyond rot_dim, two neighbouring chunks that are
// not turned.  TPH lanes (a power of two) hold a head, and its sum of squares
// is a butterfly over them: no shuffles for the rotation.
//
// cos and sin are the same for all heads of a token: a block works on U
// tokens and all heads of a group, its threads make each token's R / 2 angles
// once, into shared memory, while the heads' loads are in flight.

template <class T>
struct Chunk {
    static constexpr int kElems = 16 / T::kBytes;
};

using rmsn::F2;

// One 16-byte chunk as its four words, and as pairs of neighbouring elements.
struct Words {
    uint32_t u[4];
};
__device__ __forceinline__ Words words(const uint4& v) { return {{v.x, v.y, v.z, v.w}}; }

template <class T>
__device__ __forceinline__ void widen(const Words& w, F2 (&y)[8 / T::kBytes]) {
    if constexpr (T::kBytes == 4) {
        y[0] = rmsn::f2(__uint_as_float(w.u[0]), __uint_as_float(w.u[1]));
        y[1] = rmsn::f2(__uint_as_float(w.u[2]), __uint_as_float(w.u[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = rmsn::widen2<T>(w.u[k]);
    }
}
template <class T>
__device__ __forceinline__ float sum_squares(const Words& w, float acc) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (T::kBytes == 4) {
            const float x = __uint_as_float(w.u[k]);
            acc = fmaf(x, x, acc);
        } else {
            acc = rmsn::sumsq16x2<T>(w.u[k], acc);
        }
    }
    return acc;
}
// y = (w + woff) * (x * inv).  Without an offset the 16-bit product x w is
// exact in fp32 and goes into the FMA unwidened: y = RN((x w) inv).
template <class T>
__device__ __forceinline__ void normed(const Words& x, const Words& w, float inv, float woff,
                                       F2 (&y)[8 / T::kBytes]) {
    const F2 inv2 = rmsn::f2(inv, inv);
    if constexpr (T::kBytes == 2) {
        if (woff == 0.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                y[k] = rmsn::mul2(rmsn::mul16x2_exact<T>(x.u[k], w.u[k]), inv2);
            return;
        }
    }
    F2 v[8 / T::kBytes];
    widen<T>(x, y);
    widen<T>(w, v);
#pragma unroll
    for (int k = 0; k < 8 / T::kBytes; ++k)
        y[k] = rmsn::mul2(rmsn::add2(v[k], rmsn::f2(woff, woff)), rmsn::mul2(y[k], inv2));
}
template <class T>
__device__ __forceinline__ void store_chunk(char* p, const F2 (&y)[8 / T::kBytes]) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 8 / T::kBytes; ++k) {
        float lo, hi;
        rmsn::f2split(y[k], lo, hi);
        if constexpr (T::kBytes == 4) {
            u[2 * k] = __float_as_uint(lo);
            u[2 * k + 1] = __float_as_uint(hi);
        } else {
            u[k] = rmsn::pack2<T>(lo, hi);
        }
    }
    rmsn::st_stream16(p, u);
}
__device__ __forceinline__ void lds_f2x2(const float* p, F2& a, F2& b) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    a = rmsn::f2(v.x, v.y);
    b = rmsn::f2(v.z, v.w);
}

// Multi-head, U tokens a block.  Warp w of block (b, y) holds heads
// (y W + w) NH .. + NH - 1 (NH = 32 / TPH, W warps) of tokens b U .. + U - 1.
// Bound to 48 registers, so that 40 warps share an SM: every warp waits once
// for the block's angles, and the others' loads have to fill that time.  On a
// GB300, 16384 tokens x 40 heads x 128 bf16 (335.7 MB): 54 us with two tokens
// a block, 57 at 64 registers, 55 with three or four tokens, 61 and 83 where
// each warp makes its own angles for 8 or 4 heads and nothing waits.
template <class T, int TPH, int U, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32, 40 / kRopeWarps) rope_vec(const RopeArgs a) {
    constexpr int VE = Chunk<T>::kElems;  // elements of a chunk
    constexpr int NP = VE / 2;            // F2 of a chunk
    constexpr int NH = 32 / TPH;
    // per token R / 2 cosines, then as many sines, in fours: four of lane 0,
    // four of lane 1, ...; a warp's 16-byte reads fall on different banks
    extern __shared__ __align__(16) float cs_all[];
    rmsn::pdl_launch_dependents(a.pdl);
    const int lane = threadIdx.x & 31, sub = lane % TPH;
    const int hh = ((int)blockIdx.y * (int)(blockDim.x >> 5) + (int)(threadIdx.x >> 5)) * NH + lane / TPH;
    const bool is_q = hh < a.Hq;
    const bool on = hh < a.Hq + a.Hk && sub * 2 * VE < a.D;
    // this lane's chunks: elements [e0, e0 + VE) and [e1, e1 + VE) of the head
    const int turned = a.R / (2 * VE);  // lanes whose chunks are turned
    const bool rot = sub < turned;
    const int e0 = rot ? sub * VE : a.R + (sub - turned) * 2 * VE;
    const int e1 = rot ? a.R / 2 + sub * VE : e0 + VE;
    const int h = is_q ? hh : hh - a.Hq;
    const int64_t ss = is_q ? a.qs : a.ks, ds = is_q ? a.qos : a.kos;
    const char* src = static_cast<const char*>(is_q ? a.q : a.k) + (int64_t)h * a.D * T::kBytes;
    char* dst = static_cast<char*>(is_q ? a.qo : a.ko) + (int64_t)h * a.D * T::kBytes;
    const char* w = static_cast<const char*>(is_q ? a.qw : a.kw);
    const int P = a.R / 2;
    rmsn::pdl_wait(a.pdl);
    const int64_t t0 = (int64_t)blockIdx.x * U;
    uint4 x0[U], x1[U];
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        x0[j] = x1[j] = make_uint4(0u, 0u, 0u, 0u);
        if (on && t0 + j < a.T) {
            const char* p = src + (t0 + j) * ss * T::kBytes;
            x0[j] = rmsn::ld_stream16(p + e0 * T::kBytes);
            x1[j] = rmsn::ld_stream16(p + e1 * T::kBytes);
        }
    }
    if (a.norm && on) {
        if (w) {
            w0 = rmsn::ld_keep16(w + e0 * T::kBytes);
            w1 = rmsn::ld_keep16(w + e1 * T::kBytes);
        } else {
            const uint32_t one = rmsn::ones_word<T>();
            w0 = w1 = make_uint4(one, one, one, one);
        }
    }
    for (int i = threadIdx.x; i < U * P; i += blockDim.x) {
        const int j = i / P, p = i - j * P;
        if (t0 + j >= a.T) continue;
        const float2 cs = turn(a, p, t0 + j);
        // lane and place of the pair among the lane's VE pairs
        int s, k;
        if constexpr (INTER) {  // NP pairs of the first chunk, NP of the second
            const int half = P / 2, q = p < half ? p : p - half;
            s = q / NP;
            k = q % NP + (p < half ? 0 : NP);
        } else {
            s = p / VE;
            k = p % VE;
        }
        float* c = cs_all + j * 2 * P + ((k >> 2) * turned + s) * 4 + (k & 3);
        c[0] = cs.x;
        c[P] = cs.y;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < U; ++j) {
        F2 y0[NP], y1[NP];
        if (a.norm) {
            float acc = sum_squares<T>(words(x1[j]), sum_squares<T>(words(x0[j]), 0.f));
#pragma unroll
            for (int o = TPH / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
            const float inv = __frsqrt_rn(__fadd_rn(
                a.rcp_d > 0.f ? __fmul_rn(acc, a.rcp_d) : __fdiv_rn(acc, (float)a.D), a.eps));
            normed<T>(words(x0[j]), words(w0), inv, a.woff, y0);
            normed<T>(words(x1[j]), words(w1), inv, a.woff, y1);
        } else {
            widen<T>(words(x0[j]), y0);
            widen<T>(words(x1[j]), y1);
        }
        if (!on || t0 + j >= a.T) continue;
        if (rot) {
            const float* cs = cs_all + j * 2 * P + sub * 4;
#pragma unroll
            for (int k = 0; k < VE / 4; ++k) {  // four pairs
                F2 c[2], s[2];
                lds_f2x2(cs + k * turned * 4, c[0], c[1]);
                lds_f2x2(cs + P + k * turned * 4, s[0], s[1]);
                if constexpr (INTER) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        F2& y = 4 * k + i < NP ? y0[(4 * k + i) % NP] : y1[(4 * k + i) % NP];
                        float cl[2], sl[2], p, q;
                        rmsn::f2split(c[i >> 1], cl[0], cl[1]);
                        rmsn::f2split(s[i >> 1], sl[0], sl[1]);
                        rmsn::f2split(y, p, q);
                        y = rmsn::f2(p * cl[i & 1] - q * sl[i & 1], q * cl[i & 1] + p * sl[i & 1]);
                    }
                } else {
                    const F2 neg = rmsn::f2(-1.f, -1.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 p = y0[2 * k + i], q = y1[2 * k + i];
                        y0[2 * k + i] = rmsn::fma2(q, rmsn::mul2(s[i], neg), rmsn::mul2(p, c[i]));
                        y1[2 * k + i] = rmsn::fma2(p, s[i], rmsn::mul2(q, c[i]));
                    }
                }
            }
        }
        char* p = dst + (t0 + j) * ds * T::kBytes;
        store_chunk<T>(p + e0 * T::kBytes, y0);
        store_chunk<T>(p + e1 * T::kBytes, y1);
    }
}

#define ROPE_T(T, DT, TPH, U)                                                       \
    {DT, TPH, U, 0, (const void*)&rope_vec<T, TPH, U, false>},                      \
        {DT, TPH, U, 1, (const void*)&rope_vec<T, TPH, U, true>}
#define ROPE_D(T, DT)                                                               \
    ROPE_T(T, DT, 1, 1), ROPE_T(T, DT, 2, 1), ROPE_T(T, DT, 4, 1), ROPE_T(T, DT, 8, 1), \
        ROPE_T(T, DT, 16, 1), ROPE_T(T, DT, 32, 1), ROPE_T(T, DT, 1, 2),            \
        ROPE_T(T, DT, 2, 2), ROPE_T(T, DT, 4, 2), ROPE_T(T, DT, 8, 2),              \
        ROPE_T(T, DT, 16, 2), ROPE_T(T, DT, 32, 2)

const RopeEntry* rope_kernels(int* n) {
    static const RopeEntry table[] = {ROPE_D(F32, 0), ROPE_D(BF16, 1), ROPE_D(F16, 2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

const void* rope_generic_kernel(int dt) {
    return dt == 0 ? (const void*)&rope_generic<F32>
                   : (dt == 1 ? (const void*)&rope_generic<BF16> : (const void*)&rope_generic<F16>);
}

}  // namespace rmsattn
