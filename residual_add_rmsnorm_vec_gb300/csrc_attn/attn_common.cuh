// Device helpers of the attention-path kernels.
#pragma once

#include "../csrc/rmsn_kernels.cuh"
#include "attn_args.h"

namespace rmsattn {

using rmsn::BF16;
using rmsn::F16;
using rmsn::F32;

// One element of a T array as float, and back (rounded to nearest even).
template <class T>
__device__ __forceinline__ float load1(const void* p, int64_t e) {
    if constexpr (T::kBytes == 4) {
        return static_cast<const float*>(p)[e];
    } else {
        return rmsn::lo2<T>(static_cast<const uint16_t*>(p)[e]);
    }
}
template <class T>
__device__ __forceinline__ void store1(void* p, int64_t e, float v) {
    if constexpr (T::kBytes == 4) static_cast<float*>(p)[e] = v;
    else static_cast<uint16_t*>(p)[e] = (uint16_t)(rmsn::pack2<T>(v, 0.f) & 0xFFFFu);
}

// Two floats to E4M3 (nearest even, saturating), lo in the low byte; NaN gives
// the NaN code.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// The two E4M3 codes in the low half of u, exactly, as packed fp16 (every
// E4M3 value is an fp16 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t u) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)u));
    return d;
}

// Page of token j of a table row, or -1 where the table or the cache ends.
__device__ __forceinline__ int64_t page_of(const Cache& c, const int32_t* row, int64_t width,
                                           int64_t j) {
    const int64_t slot = j / c.page;
    if (slot >= width) return -1;
    const int64_t p = row[slot];
    return p >= 0 && p < c.n_pages ? p : -1;
}

}  // namespace rmsattn
