// Attention of a group's queries over the tokens that the group shares: the parts
// that attn_attend.cuh's kernels add to each sequence's own tokens.
//
// A row is one column of the group (sequence x query token x head of a key head);
// four threads to a row, a quarter of the dims each.
#include "attn_common.cuh"

namespace rmsattn {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -3.402823466e38f;

template <class T, int D>
__global__ void __launch_bounds__(256) prefix_kernel(const PrefixArgs a) {
    constexpr int Q = D / 4;
    __shared__ float ks[kBlock][D], vs[kBlock][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const PrefixLine line = *a.line;
    const int begin = blockIdx.x * line.chunk;
    const int stop = begin + line.chunk < line.total ? begin + line.chunk : line.total;
    const int quarter = threadIdx.x & 3, r0 = threadIdx.x >> 2;
    int g = 0;
    for (int at = begin; at < stop;) {
        while (at >= a.groups[g].first + a.groups[g].ns * a.groups[g].tiles * a.c.H) ++g;
        const PrefixGroup G = a.groups[g];
        const int item = (at - G.first) / G.ns, step0 = (at - G.first) % G.ns;
        const int steps = stop - at < G.ns - step0 ? stop - at : G.ns - step0;
        const int hk = item / G.tiles, tile = item % G.tiles;
        const int cols = (G.s1 - G.s0) * a.n * a.group;
        float* part = a.parts + (blockIdx.x + G.item0 + item) * prefix_part(D);
        for (int half = 0; half < kPrefixRows; half += 64) {
            const int row = half + r0, cc = tile * kPrefixRows + row;
            const bool on = cc < cols;
            float q[Q], o[Q], m = kNone, l = 0.f;
            const int64_t token = (int64_t)G.s0 * a.n + cc / a.group;
            const int64_t qe = token * a.q_stride + (int64_t)(hk * a.group + cc % a.group) * D + quarter * Q;
#pragma unroll
            for (int d = 0; d < Q; ++d) {
                q[d] = on ? load1<T>(a.q, qe + d) * (a.scale * kLog2e) : 0.f;
                o[d] = 0.f;
            }
            const int t1 = (step0 + steps) * a.tok < G.shared ? (step0 + steps) * a.tok : G.shared;
            for (int t0 = step0 * a.tok; t0 < t1; t0 += kBlock) {
                const int64_t page = page_of(a.c, a.table + G.seq * a.table_stride, a.table_width, t0);
                if (page < 0) {
                    if (threadIdx.x == 0) atomicOr(a.status, kBadPage);
                    continue;
                }
                const int blk = hk * (a.c.page / kBlock) + t0 % a.c.page / kBlock;
                const int64_t codes = page * a.c.page_stride + (int64_t)blk * kBlock * D;
                const float fk = a.c.ks[page * a.c.scale_stride + blk], fv = a.c.vs[page * a.c.scale_stride + blk];
                __syncthreads();
                for (int e = threadIdx.x; e < kBlock * D; e += 256) {
                    ks[e / D][e % D] = rmsn::e4m3_value(a.c.k[codes + e]) * fk;
                    vs[e / D][e % D] = rmsn::e4m3_value(a.c.v[codes + e]) * fv;
                }
                __syncthreads();
                for (int j = 0; j < kBlock; ++j) {
                    float s = 0.f;
#pragma unroll
                    for (int d = 0; d < Q; ++d) s = fmaf(q[d], ks[j][quarter * Q + d], s);
                    s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
                    s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
                    const float to = fmaxf(m, s), keep = exp2f(m - to), p = exp2f(s - to);
                    m = to;
                    l = l * keep + p;
#pragma unroll
                    for (int d = 0; d < Q; ++d) o[d] = fmaf(o[d], keep, p * vs[j][quarter * Q + d]);
                }
            }
            if (on) {
#pragma unroll
                for (int d = 0; d < Q; ++d) {
                    const int dd = quarter * Q + d;
                    part[(dd / 8 * kPrefixRows + row) * 8 + dd % 8] = o[d];
                }
                if (quarter == 0) {
                    part[D * kPrefixRows + row * 2] = m;
                    part[D * kPrefixRows + row * 2 + 1] = l;
                }
            }
        }
        at += steps;
    }
}

template <class T, int D>
PrefixEntry entry(int dt) {
    return PrefixEntry{dt, D, D == 256 ? 64 : 128, 256, 0, (const void*)&prefix_kernel<T, D>};
}

}  // namespace

const PrefixEntry* prefix_kernels(int* n) {
    static const PrefixEntry table[] = {entry<BF16, 64>(1),  entry<F16, 64>(2),  entry<BF16, 128>(1),
                                        entry<F16, 128>(2), entry<BF16, 256>(1), entry<F16, 256>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
