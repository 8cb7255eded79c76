// Attention over the paged E4M3 cache.
//
//   s_j = scale q . k_j,  m = max s_j,  out = sum exp(s_j - m) v_j / sum exp(s_j - m)
//
// in one pass over the tokens: m, the sum l and the weighted sum are carried
// along, and multiplied by exp(m_old - m_new) where the maximum grows.
#include "attn_common.cuh"

namespace rmsattn {

// One warp per sequence, query and query head; 32 tokens at a time.
template <class T>
__global__ void __launch_bounds__(128) attend_simple(const AttendArgs a) {
    __shared__ float qs[4][256];
    rmsn::pdl_launch_dependents(a.pdl);
    rmsn::pdl_wait(a.pdl);
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t u = (int64_t)blockIdx.x * 4 + wp;
    if (u >= a.B * a.n * a.Hq) return;
    const int64_t b = u / ((int64_t)a.n * a.Hq);
    const int i = (int)(u / a.Hq % a.n), h = (int)(u % a.Hq);
    const int D = a.c.D, hk = h / (a.Hq / a.c.H);
    const int64_t row = b * a.n + i;
    for (int d = lane; d < D; d += 32)
        qs[wp][d] = load1<T>(a.q, row * a.q_stride + (int64_t)h * D + d);
    __syncwarp();
    const int64_t pos = (int64_t)a.lengths[b] - a.n + i;
    const int64_t room = a.table_width * a.c.page;
    if (pos >= room && lane == 0) atomicOr(a.status, kBadPage);
    const int32_t* table = a.table + b * a.table_stride;
    float m = -INFINITY, l = 0.f, o[8];
    for (int d = 0; d < 8; ++d) o[d] = 0.f;
    for (int64_t j0 = 0; j0 <= pos && j0 < room; j0 += 32) {
        const int64_t j = j0 + lane;
        bool seen = j <= pos && (a.window == 0 || j > pos - a.window || j < a.sinks);
        if (!__any_sync(0xFFFFFFFFu, seen)) continue;
        int64_t at = 0;
        float ks = 0.f, vs = 0.f, s = -INFINITY;
        if (seen) {
            const int64_t pg = page_of(a.c, table, a.table_width, j);
            if (pg < 0) {
                seen = false;
                atomicOr(a.status, kBadPage);
            } else {
                const int64_t in = j % a.c.page;
                at = pg * a.c.page_stride + ((int64_t)hk * a.c.page + in) * D;
                const int64_t sc = pg * a.c.scale_stride + (int64_t)hk * (a.c.page / kBlock) +
                                   in / kBlock;
                ks = a.c.ks[sc];
                vs = a.c.vs[sc];
            }
        }
        if (seen) {
            float acc = 0.f;
            for (int d = 0; d < D; ++d)
                acc = fmaf(qs[wp][d], rmsn::e4m3_value(a.c.k[at + d]), acc);
            s = acc * ks * a.scale;
        }
        float mj = s;
        for (int k = 16; k > 0; k >>= 1) mj = fmaxf(mj, __shfl_xor_sync(0xFFFFFFFFu, mj, k));
        const float mn = fmaxf(m, mj), ms = mn == -INFINITY ? 0.f : mn;
        const float keep = expf(m - ms), p = expf(s - ms);
        m = mn;
        l = l * keep + rmsn::warp_sum(p);
        for (int d = 0; d < 8; ++d) o[d] *= keep;
        for (int k = 0; k < 32; ++k) {
            const bool on = __shfl_sync(0xFFFFFFFFu, (int)seen, k);
            const float pk = __shfl_sync(0xFFFFFFFFu, p * vs, k);
            const int64_t ak = __shfl_sync(0xFFFFFFFFu, at, k);
            if (!on) continue;
            for (int d = 0; d < 8 && d * 32 < D; ++d)
                o[d] = fmaf(pk, rmsn::e4m3_value(a.c.v[ak + d * 32 + lane]), o[d]);
        }
    }
    for (int d = 0; d < 8 && d * 32 < D; ++d)
        store1<T>(a.out, row * a.out_stride + (int64_t)h * D + d * 32 + lane,
                  l == 0.f ? 0.f : o[d] / l);
}

const void* attend_simple_kernel(int dt) {
    return dt == 1 ? (const void*)&attend_simple<BF16> : (const void*)&attend_simple<F16>;
}

}  // namespace rmsattn
