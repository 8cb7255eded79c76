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

template <class T>
__device__ __forceinline__ void unpack16(const uint4& v, float (&x)[16 / T::kBytes]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (T::kBytes == 4) {
            x[k] = __uint_as_float(u[k]);
        } else {
            x[2 * k] = rmsn::lo2<T>(u[k]);
            x[2 * k + 1] = rmsn::hi2<T>(u[k]);
        }
    }
}
template <class T>
__device__ __forceinline__ uint4 pack16(const float (&x)[16 / T::kBytes]) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (T::kBytes == 4) u[k] = __float_as_uint(x[k]);
        else u[k] = rmsn::pack2<T>(x[2 * k], x[2 * k + 1]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Multi-head, U tokens a block.  Warp w of block (b, y) holds heads
// (y W + w) NH .. + NH - 1 (NH = 32 / TPH, W warps) of tokens b U .. + U - 1.
template <class T, int TPH, int U, bool INTER>
__global__ void __launch_bounds__(512) rope_vec(const RopeArgs a) {
    constexpr int VE = Chunk<T>::kElems;  // elements of a chunk
    constexpr int NH = 32 / TPH;
    // [U][R / 2] (cos, sin), element k of all lanes' chunks side by side: a
    // warp's reads of it fall on different banks
    extern __shared__ float2 cs_all[];
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
    const char* src = static_cast<const char*>(is_q ? a.q : a.k);
    char* dst = static_cast<char*>(is_q ? a.qo : a.ko);
    const int64_t ss = is_q ? a.qs : a.ks, ds = is_q ? a.qos : a.kos;
    const char* w = static_cast<const char*>(is_q ? a.qw : a.kw);
    const int P = a.R / 2;
    rmsn::pdl_wait(a.pdl);
    const int64_t t0 = (int64_t)blockIdx.x * U;
    uint4 x0[U], x1[U], w0, w1;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if (on && t0 + j < a.T) {
            const char* p = src + ((t0 + j) * ss + (int64_t)h * a.D) * T::kBytes;
            x0[j] = rmsn::ld_stream16(p + e0 * T::kBytes);
            x1[j] = rmsn::ld_stream16(p + e1 * T::kBytes);
        } else {
            x0[j] = x1[j] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    const bool weighted = a.norm && w != nullptr && on;
    if (weighted) {
        w0 = rmsn::ld_keep16(w + e0 * T::kBytes);
        w1 = rmsn::ld_keep16(w + e1 * T::kBytes);
    }
    for (int i = threadIdx.x; i < U * P; i += blockDim.x) {
        const int64_t t = t0 + i / P;
        if (t >= a.T) continue;
        const int p = i % P;
        int at;
        if constexpr (INTER) {
            const int half = P / 2, q = p % half;
            at = p - q + (q % (VE / 2)) * turned + q / (VE / 2);
        } else {
            at = (p % VE) * turned + p / VE;
        }
        cs_all[i - p + at] = turn(a, p, t);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < U; ++j) {
        float y0[VE], y1[VE];
        unpack16<T>(x0[j], y0);
        unpack16<T>(x1[j], y1);
        if (a.norm) {
            float acc = 0.f;
#pragma unroll
            for (int k = 0; k < VE; ++k) acc = fmaf(y0[k], y0[k], acc);
#pragma unroll
            for (int k = 0; k < VE; ++k) acc = fmaf(y1[k], y1[k], acc);
#pragma unroll
            for (int o = TPH / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
            const float inv = __frsqrt_rn(__fadd_rn(
                a.rcp_d > 0.f ? __fmul_rn(acc, a.rcp_d) : __fdiv_rn(acc, (float)a.D), a.eps));
            float v0[VE], v1[VE];
            if (weighted) {
                unpack16<T>(w0, v0);
                unpack16<T>(w1, v1);
            } else {
#pragma unroll
                for (int k = 0; k < VE; ++k) v0[k] = v1[k] = 1.f;
            }
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                y0[k] = (v0[k] + a.woff) * (y0[k] * inv);
                y1[k] = (v1[k] + a.woff) * (y1[k] * inv);
            }
        }
        if (!on || t0 + j >= a.T) continue;
        if (rot) {
            const float2* cs = cs_all + j * P;
            if constexpr (INTER) {
                // pairs e / 2 of both chunks
#pragma unroll
                for (int k = 0; k < VE / 2; ++k) {
                    const float2 c0 = cs[k * turned + sub], c1 = cs[P / 2 + k * turned + sub];
                    const float p0 = y0[2 * k], q0 = y0[2 * k + 1], p1 = y1[2 * k], q1 = y1[2 * k + 1];
                    y0[2 * k] = p0 * c0.x - q0 * c0.y;
                    y0[2 * k + 1] = q0 * c0.x + p0 * c0.y;
                    y1[2 * k] = p1 * c1.x - q1 * c1.y;
                    y1[2 * k + 1] = q1 * c1.x + p1 * c1.y;
                }
            } else {
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    const float2 c = cs[k * turned + sub];
                    const float p = y0[k], q = y1[k];
                    y0[k] = p * c.x - q * c.y;
                    y1[k] = q * c.x + p * c.y;
                }
            }
        }
        char* p = dst + ((t0 + j) * ds + (int64_t)h * a.D) * T::kBytes;
        const uint4 o0 = pack16<T>(y0), o1 = pack16<T>(y1);
        rmsn::st_stream16(p + e0 * T::kBytes, &o0.x);
        rmsn::st_stream16(p + e1 * T::kBytes, &o1.x);
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
