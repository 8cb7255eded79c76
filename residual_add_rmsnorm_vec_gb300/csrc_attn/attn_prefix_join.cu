// Attention with a shared prefix: the parts of a row, those of its group's shared tokens
// in the order of the line's shares, and that of its own tokens:
//
//   out = sum_i O_i 2^(m_i - m) / sum_i l_i 2^(m_i - m),  m = max m_i
//
// What bounds it: the chain of loads (sequence, group, parts) and the parts' bytes from
// L2.  A thread has eight dims of a row and every fourth part where there are many (else
// all of them), up to eight of them on their
// way at once; lanes run along a key head's columns, as those lie in the parts (32
// bytes each).  64 sequences of 32 / 8 heads x 128 with 19 parts 8 us, 256 with 6 parts 13 us;
// with the dims along the lanes and one thread to all parts, the former took 17 us.
#include "attn_common.cuh"

namespace rmsattn {

namespace {

constexpr float kNone = -3.402823466e38f;

__device__ __forceinline__ float exp2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void add(float4& y, const float4& v, float f) {
    y.x += v.x * f;
    y.y += v.y * f;
    y.z += v.z * f;
    y.w += v.w * f;
}

// kWays threads to a row's parts.  Four blocks of four ways to an SM, for 64 sequences x 8192
// then join in one wave (512 blocks; at 70 registers, three to an SM, 55.8 us and not 52.8).
template <class T, int kWays>
__global__ void __launch_bounds__(256, kWays == 4 ? 4 : 3) prefix_join(const PrefixJoinArgs a) {
    constexpr int kCols = 256 / kWays;
    __shared__ float4 sum[kWays][2][kCols];
    __shared__ float2 ref[kWays][kCols];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x % kCols, way = threadIdx.x / kCols;
    const int64_t cols = a.rows / a.Hq * a.group;
    int64_t col = blockIdx.x * (int64_t)kCols + lane;
    const bool on = col < cols;
    if (!on) col = cols - 1;
    const int hk = blockIdx.y / (a.D / 8), d = blockIdx.y % (a.D / 8) * 8;
    const int64_t token = col / a.group, b = token / a.n;
    const int head = hk * a.group + (int)(col - token * a.group);
    const int64_t row = token * a.Hq + head;
    const PrefixSeq sq = a.seqs[b];
    PrefixGroup g = a.groups[0];  // (on its way with the sequence's word)
    const uint32_t chunk = a.line->chunk;
    float m = kNone, l = 0.f;
    float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f), y1 = y0;
    if (way == 0) {
        const float2 own = a.own_ml[row];
        const float4* o = reinterpret_cast<const float4*>(a.own + row * a.D + d);
        y0 = o[0];
        y1 = o[1];
        m = own.x;
        l = own.y;
    }
    if (sq.start > 0) {
        if (sq.group > 0) g = a.groups[sq.group];
        const int cc = ((int)(token - (int64_t)g.s0 * a.n)) * a.group + head - hk * a.group;
        const int tile = cc / a.item_rows, r = cc - tile * a.item_rows, item = hk * g.tiles + tile;
        const uint32_t at = (uint32_t)g.first + (uint32_t)item * (uint32_t)g.ns;
        const int first = (int)(at / chunk), n = (int)((at + (uint32_t)g.ns - 1) / chunk) - first + 1;
        const uint32_t eight = first * (a.item_rows / 8) + (r >> 3) + prefix_eight(g, a.n * a.group, hk, tile, a.item_rows);
        const int size = a.item_rows * (a.D + 2);  // from a share's part to the next one's
        const float* p = a.parts + (int64_t)eight * (8 * (a.D + 2)) + d * 8 + (r & 7) * 8;
        const int to_ml = (a.D - d) * 8 - (r & 7) * 6;
        constexpr int U = 8;
        for (int k0 = way; k0 < n; k0 += U * kWays) {
            float2 ml[U];
            float4 v[U][2];
#pragma unroll
            for (int k = 0; k < U; ++k) {  // (past the last: the last again, not added)
                const float* q = p + (k0 + k * kWays < n ? k0 + k * kWays : n - 1) * size;
                ml[k] = *reinterpret_cast<const float2*>(q + to_ml);
                v[k][0] = *reinterpret_cast<const float4*>(q);
                v[k][1] = *reinterpret_cast<const float4*>(q + 4);
            }
            float to = m;
#pragma unroll
            for (int k = 0; k < U; ++k) to = fmaxf(to, ml[k].x);
            const float keep = exp2a(m - to);
            m = to;
            l *= keep;
            y0 = make_float4(y0.x * keep, y0.y * keep, y0.z * keep, y0.w * keep);
            y1 = make_float4(y1.x * keep, y1.y * keep, y1.z * keep, y1.w * keep);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (k0 + k * kWays >= n) break;
                const float f = exp2a(ml[k].x - m);
                l += ml[k].y * f;
                add(y0, v[k][0], f);
                add(y1, v[k][1], f);
            }
        }
    }
    sum[way][0][lane] = y0;
    sum[way][1][lane] = y1;
    ref[way][lane] = make_float2(m, l);
    __syncthreads();
    if (way > 0 || !on) return;
    float2 ml[kWays];
#pragma unroll
    for (int k = 0; k < kWays; ++k) {
        ml[k] = ref[k][lane];
        m = fmaxf(m, ml[k].x);
    }
    l = 0.f;
    y0 = y1 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWays; ++k) {
        const float f = exp2a(ml[k].x - m);
        l += ml[k].y * f;
        add(y0, sum[k][0][lane], f);
        add(y1, sum[k][1][lane], f);
    }
    const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        u[k] = rmsn::pack2<T>(l == 0.f ? 0.f : y[2 * k] / l, l == 0.f ? 0.f : y[2 * k + 1] / l);
    uint16_t* out = static_cast<uint16_t*>(a.out) + token * a.out_stride + (int64_t)head * a.D + d;
    *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace

const void* prefix_join_kernel(int dt, int ways) {
    if (ways == 1) return dt == 1 ? (const void*)&prefix_join<BF16, 1> : (const void*)&prefix_join<F16, 1>;
    return dt == 1 ? (const void*)&prefix_join<BF16, 4> : (const void*)&prefix_join<F16, 4>;
}

}  // namespace rmsattn
