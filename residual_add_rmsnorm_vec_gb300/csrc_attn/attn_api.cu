// C ABI of the attention-path operators (include/rmsnorm_attn.h): argument
// checks, launch shapes and launches.
#include <math.h>
#include <string.h>

#include "attn_host.h"

namespace rmsattn {
namespace {

// Status word of the kernels on each device.
__device__ uint32_t g_status;

DeviceInfo g_dev[kMaxDevices];

}  // namespace

DeviceInfo* device_info() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    DeviceInfo& d = g_dev[dev];
    std::call_once(d.once, [&] {
        d.err = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (d.err == cudaSuccess) d.err = cudaGetSymbolAddress((void**)&d.status, g_status);
    });
    return d.err == cudaSuccess ? &d : nullptr;
}

int launch(const void* fn, dim3 grid, int threads, size_t smem, void* args, bool pdl,
           cudaStream_t stream, int cluster) {
    void* list[] = {args};
    if (!pdl && cluster == 1)
        return cudaLaunchKernel(fn, grid, dim3(threads), list, smem, stream) == cudaSuccess
                   ? RMSN_OK
                   : RMSN_ECUDA;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = n;
    return cudaLaunchKernelExC(&lc, fn, list) == cudaSuccess ? RMSN_OK : RMSN_ECUDA;
}

int check_cache(const rmsattn_cache* c, Cache* out) {
    if (!c || c->reserved != 0) return RMSN_EINVAL;
    if (c->n_pages < 0 || c->n_pages > INT32_MAX || c->n_kv_heads < 1 || c->n_kv_heads > 4096)
        return RMSN_EINVAL;
    if (c->page_size < kBlock || c->page_size > 65536 || c->page_size % kBlock) return RMSN_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return RMSN_EUNSUPPORTED;
    const int64_t codes = (int64_t)c->n_kv_heads * c->page_size * c->head_dim;
    const int64_t scales = (int64_t)c->n_kv_heads * (c->page_size / kBlock);
    if (c->page_stride < codes || c->page_stride % 16 || c->scale_stride < scales)
        return RMSN_EINVAL;
    if (too_big(times(c->n_pages, c->page_stride)) || too_big(times(c->n_pages, c->scale_stride)))
        return RMSN_EINVAL;
    // a scale's place is counted in 32 bits
    if (times(c->n_pages, c->scale_stride) >= (int64_t(1) << 32)) return RMSN_EUNSUPPORTED;
    if (c->n_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return RMSN_EINVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
        !aligned(c->v_scale, 4))
        return RMSN_EALIGN;
    out->k = (uint8_t*)c->k;
    out->v = (uint8_t*)c->v;
    out->ks = c->k_scale;
    out->vs = c->v_scale;
    out->n_pages = c->n_pages;
    out->page_stride = c->page_stride;
    out->scale_stride = c->scale_stride;
    out->H = c->n_kv_heads;
    out->page = c->page_size;
    out->D = c->head_dim;
    return RMSN_OK;
}

int check_table(const int32_t* table, int64_t stride, int64_t width, int64_t n_seqs, int page) {
    if (width < 0 || stride < width || times(width, page) > kMaxTokens) return RMSN_EINVAL;
    if (too_big(times(n_seqs, stride))) return RMSN_EINVAL;
    if (n_seqs > 0 && width > 0 && !table) return RMSN_EINVAL;
    return aligned(table, 4) ? RMSN_OK : RMSN_EALIGN;
}

}  // namespace rmsattn

using namespace rmsattn;

RMSATTN_API int rmsattn_qk_rope_fwd(const void* q, const void* k, const void* q_weight,
                                    const void* k_weight, void* q_out, void* k_out,
                                    const void* positions, int64_t pos_stride,
                                    const uint64_t* turns, const int32_t* axis, int64_t n_tokens,
                                    int64_t n_q_heads, int64_t n_k_heads, int64_t head_dim,
                                    int64_t rot_dim, int64_t n_axes, int64_t q_stride,
                                    int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                                    float eps, float weight_offset, uint32_t flags,
                                    cudaStream_t stream) {
    if (flags & ~(RMSN_IN_MASK | RMSN_PDL | RMSATTN_NORM | RMSATTN_INTERLEAVED | RMSATTN_POS_I64))
        return RMSN_EINVAL;
    int64_t bytes = 0;
    const int dt = dtype_of(flags, &bytes);
    if (dt < 0) return RMSN_EINVAL;
    if (n_tokens < 0 || n_q_heads < 0 || n_k_heads < 0 || head_dim < 1 || head_dim > 4096)
        return RMSN_EINVAL;
    if (n_q_heads > (1 << 20) || n_k_heads > (1 << 20)) return RMSN_EINVAL;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 || n_axes < 0 || n_axes > 64)
        return RMSN_EINVAL;
    if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(weight_offset)) return RMSN_EINVAL;
    if (n_q_heads && (q_stride < n_q_heads * head_dim || q_out_stride < n_q_heads * head_dim))
        return RMSN_EINVAL;
    if (n_k_heads && (k_stride < n_k_heads * head_dim || k_out_stride < n_k_heads * head_dim))
        return RMSN_EINVAL;
    const int64_t strides[] = {n_q_heads ? q_stride : 0, n_q_heads ? q_out_stride : 0,
                               n_k_heads ? k_stride : 0, n_k_heads ? k_out_stride : 0};
    for (int64_t s : strides)
        if (too_big(times(n_tokens, times(s, 4)))) return RMSN_EINVAL;
    if (rot_dim && (n_axes < 1 || pos_stride < 0 || too_big(times(n_axes, times(pos_stride, 8)))))
        return RMSN_EINVAL;
    // 0: one row serves every axis (text among images)
    if (n_axes > 1 && pos_stride != 0 && pos_stride < n_tokens) return RMSN_EINVAL;
    if (n_tokens == 0 || n_q_heads + n_k_heads == 0) return RMSN_OK;
    if ((n_q_heads && (!q || !q_out)) || (n_k_heads && (!k || !k_out))) return RMSN_EINVAL;
    if (rot_dim && (!positions || !turns || !axis)) return RMSN_EINVAL;
    const void* ptrs[] = {q, k, q_weight, k_weight, q_out, k_out};
    for (const void* p : ptrs)
        if (!aligned(p, (uintptr_t)bytes)) return RMSN_EALIGN;
    if (rot_dim && (!aligned(positions, flags & RMSATTN_POS_I64 ? 8 : 4) || !aligned(turns, 8) ||
                    !aligned(axis, 4)))
        return RMSN_EALIGN;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    RopeArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.qw = q_weight;
    a.kw = k_weight;
    a.qo = q_out;
    a.ko = k_out;
    a.pos = positions;
    a.turns = turns;
    a.axis = axis;
    a.T = n_tokens;
    a.pos_stride = pos_stride;
    a.qs = q_stride;
    a.ks = k_stride;
    a.qos = q_out_stride;
    a.kos = k_out_stride;
    a.Hq = (int32_t)n_q_heads;
    a.Hk = (int32_t)n_k_heads;
    a.D = (int32_t)head_dim;
    a.R = (int32_t)rot_dim;
    a.n_axes = (int32_t)n_axes;
    a.norm = (flags & RMSATTN_NORM) ? 1 : 0;
    a.interleaved = (flags & RMSATTN_INTERLEAVED) ? 1 : 0;
    a.pos64 = (flags & RMSATTN_POS_I64) ? 1 : 0;
    a.pdl = (flags & RMSN_PDL) ? 1 : 0;
    a.eps = eps;
    a.woff = weight_offset;
    a.rcp_d = (head_dim & (head_dim - 1)) == 0 ? 1.0f / (float)head_dim : 0.f;

    // 16-byte vectors: whole chunk pairs in the head and in its turned part,
    // every head of every operand on a 16-byte boundary
    const int64_t pair = 32 / bytes;  // elements of a lane's two chunks
    bool vec = head_dim % pair == 0 && rot_dim % pair == 0 && head_dim / pair <= 32 &&
               n_tokens < (int64_t(1) << 30);
    for (const void* p : ptrs) vec = vec && aligned(p, 16);
    for (int64_t s : strides) vec = vec && (s * bytes) % 16 == 0;
    if (vec) {
        int tph = 1;
        while (tph * pair < head_dim) tph *= 2;
        // two tokens a block put twice the bytes in flight per lane once
        // there are blocks enough for every SM
        const int u = n_tokens >= 4 * (int64_t)d->num_sms ? 2 : 1;
        int n = 0;
        const RopeEntry* table = rope_kernels(&n);
        const RopeEntry* e = nullptr;
        for (int i = 0; i < n; ++i)
            if (table[i].dt == dt && table[i].tph == tph && table[i].u == u &&
                table[i].interleaved == a.interleaved)
                e = &table[i];
        // warps of 32 / tph heads, split evenly over as few blocks as hold them
        const int64_t nh = 32 / tph, warps = (n_q_heads + n_k_heads + nh - 1) / nh;
        const int64_t gy = (warps + kRopeWarps - 1) / kRopeWarps;
        if (e && gy <= 65535)
            return launch(e->fn, dim3((unsigned)((n_tokens + u - 1) / u), (unsigned)gy),
                          (int)((warps + gy - 1) / gy) * 32, (size_t)(u * rot_dim / 2) * 8, &a,
                          a.pdl, stream);
    }
    int64_t blocks = (n_tokens * (n_q_heads + n_k_heads) + 7) / 8;
    if (blocks > (1 << 30)) blocks = 1 << 30;
    return launch(rope_generic_kernel(dt), dim3((unsigned)blocks), 256, 0, &a, a.pdl, stream);
}

RMSATTN_API int rmsattn_kv_append(const rmsattn_cache* cache, const void* k, const void* v,
                                  int64_t k_stride, int64_t v_stride, const int32_t* block_table,
                                  int64_t table_stride, int64_t table_width,
                                  const int32_t* lengths, const int32_t* cu_seqlens,
                                  int64_t n_tokens, int64_t n_seqs, uint32_t flags,
                                  cudaStream_t stream) {
    if (flags & ~(RMSN_IN_MASK | RMSN_PDL)) return RMSN_EINVAL;
    int64_t bytes = 0;
    const int dt = dtype_of(flags, &bytes);
    if (dt < 0) return RMSN_EINVAL;
    AppendArgs a;
    memset(&a, 0, sizeof(a));
    int st = check_cache(cache, &a.c);
    if (st != RMSN_OK) return st;
    if (n_tokens < 0 || n_seqs < 0 || n_tokens > kMaxTokens || n_seqs > (1 << 24))
        return RMSN_EINVAL;
    if (!cu_seqlens && n_tokens != n_seqs) return RMSN_EINVAL;
    const int64_t width = (int64_t)a.c.H * a.c.D;
    if (k_stride < width || v_stride < width || too_big(times(n_tokens, times(k_stride, 4))) ||
        too_big(times(n_tokens, times(v_stride, 4))))
        return RMSN_EINVAL;
    st = check_table(block_table, table_stride, table_width, n_seqs, a.c.page);
    if (st != RMSN_OK) return st;
    if (n_tokens == 0 || n_seqs == 0) return RMSN_OK;
    if (!k || !v || !lengths) return RMSN_EINVAL;
    if (!aligned(k, (uintptr_t)bytes) || !aligned(v, (uintptr_t)bytes) || !aligned(lengths, 4) ||
        !aligned(cu_seqlens, 4))
        return RMSN_EALIGN;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.lengths = lengths;
    a.cu = cu_seqlens;
    a.T = n_tokens;
    a.B = n_seqs;
    a.pdl = (flags & RMSN_PDL) ? 1 : 0;
    a.status = d->status;
    const int64_t units = cu_seqlens ? n_tokens / kBlock + 2 * n_seqs : n_seqs;
    const bool vec = aligned(k, 16) && aligned(v, 16) && (k_stride * bytes) % 16 == 0 &&
                     (v_stride * bytes) % 16 == 0;
    // a warp for each head and side of a unit, eight of them a block
    const int sides = 2 * a.c.H, warps = sides < 8 ? sides : 8;
    return launch(append_kernel_of(dt, a.c.D, vec),
                  dim3((unsigned)units, (unsigned)((sides + warps - 1) / warps)), warps * 32, 0,
                  &a, a.pdl, stream);
}

namespace rmsattn {

int check_attend(int64_t n_seqs, int64_t n_queries, int64_t n_q_heads, int64_t n_kv_heads,
                 int64_t head_dim) {
    if (n_seqs < 0 || n_seqs > (1 << 24) || n_queries < 1 || n_queries > RMSATTN_MAX_QUERIES ||
        n_kv_heads < 1 || n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % n_kv_heads)
        return RMSN_EINVAL;
    return head_dim == 64 || head_dim == 128 || head_dim == 256 ? RMSN_OK : RMSN_EUNSUPPORTED;
}

namespace {

const AttendEntry* attend_entry_of(bool behind, int dt, int64_t D, int64_t cols, int64_t tokens) {
    int n = 0;
    const AttendEntry* t = nullptr;
    if (behind)
        t = D == 64 ? attend_behind_64(&n) : (D == 128 ? attend_behind_128(&n) : attend_behind_256(&n));
    else
        t = D == 64 ? attend_kernels_64(&n) : (D == 128 ? attend_kernels_128(&n) : attend_kernels_256(&n));
    // the fewest column tiles that hold all columns, or the most there are; of
    // those the first that takes rows of so many tokens
    const AttendEntry* best = nullptr;
    for (int i = 0; i < n; ++i) {
        if (t[i].dt != dt || t[i].most < tokens) continue;
        if (!best || (best->NT * 8 < cols && t[i].NT > best->NT)) best = &t[i];
    }
    return best;
}

}  // namespace

int64_t resident_blocks(DeviceInfo* d, const void* fn, int threads, int smem, int per_sm) {
    std::lock_guard<std::mutex> lock(d->mu);
    for (int i = 0; i < d->n_resident; ++i)
        if (d->resident[i].fn == fn) return d->resident[i].blocks;
    int bps = 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&bps, fn, threads, smem) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    // no more than the shape was bounded for: both dtypes' kernels then have
    // the same grid, and so the same workspace
    const int64_t n = (int64_t)(bps < per_sm ? bps : per_sm) * d->num_sms;
    if (n > 0 && d->n_resident < 64) {
        d->resident[d->n_resident].fn = fn;
        d->resident[d->n_resident++].blocks = n;
    }
    return n;
}

int plan_attend(DeviceInfo* d, bool behind, int dt, int64_t n_seqs, int64_t n_queries, int64_t n_q_heads,
                int64_t n_kv_heads, int64_t head_dim, int64_t max_tokens, int64_t window,
                int64_t sinks, Plan* p) {
    // the most tokens that a row's queries see, borders of steps included (no
    // table holds kMaxTokens: beyond that neither limits anything, and the sum
    // stays within 64 bits)
    if (window > 0 && window < kMaxTokens && sinks < kMaxTokens &&
        window + n_queries + sinks + 256 < max_tokens)
        max_tokens = window + n_queries + sinks + 256;
    const int64_t cols = n_q_heads / n_kv_heads * n_queries;
    // A row to a cluster of `split` blocks, or the line?  The host knows the
    // tables' width, not the lengths: a long sequence among short ones keeps
    // its clusters busy alone, while the line shares everything evenly.  So
    // rows are left to clusters only while a warp's part of the longest is at
    // most 65536 / head_dim tokens (about 20 us), and then where the estimate
    // says so, measured in tokens of a warp.  A cluster's rows cost their
    // longest share times the waves of blocks; a last wave that fills part of
    // the GPU costs its part where DRAM is the bound (one column tile, head_dim
    // 128 or 256), but no less than two thirds of a full one, below which its
    // blocks wait for themselves; where instructions are the bound it costs a
    // full one.  The line costs an even share, about 5 us more (its scan and
    // its join: as long as a warp takes for 16384 / head_dim tokens), and
    // longer joins where a row has many parts.  At head_dim 128 on a GB300,
    // rows against line: 8 x 2000 tokens x 8 heads 10.6 against 14.3 us, 256 x
    // 300 38.3 against 40.4, 16 x 4000 24.7 against 27.7; and where all are as
    // long as the first, 64 x 8192 152 against 149, 1 x 131072 121 against 52.
    for (int line = 0; line < 2; ++line) {
        // the line takes the first of the fitting kernels, whatever the rows
        const AttendEntry* e = p->e = attend_entry_of(behind, dt, head_dim, cols, line ? 0 : max_tokens);
        const int64_t resident = resident_blocks(d, e->fn, e->threads, e->smem, e->per_sm);
        if (resident < 1) return RMSN_ECUDA;
        const int64_t warps = e->threads / 32;
        p->groups = (int)((cols + 8 * e->NT - 1) / (8 * e->NT));
        const int64_t rows = n_seqs * n_kv_heads * p->groups;
        const int64_t steps = max_tokens < 1 ? 1 : (max_tokens + e->tok - 1) / e->tok;
        const int64_t total = times(rows, steps);
        if (!line) {
            int64_t split = 1;
            while (split < kMaxSplit && rows * split * 2 <= resident) split *= 2;
            const double f = (double)(rows * split) / (double)resident, full = floor(f);
            const double least = e->NT == 1 && head_dim >= 128 ? 0.65 : 1.0;
            const double rest = f - full;
            const double waves = full + (rest == 0 ? 0 : (rest > least ? rest : least));
            const double part = (double)((steps + split - 1) / split) * e->tok / (double)warps;
            const double by_line = (double)total * e->tok / (double)(resident * warps) +
                                   16384.0 / (double)head_dim + 2.0 * (double)resident / (double)rows;
            if (part > 65536.0 / (double)head_dim || waves * part > by_line ||
                rows * split >= (int64_t(1) << 31))
                continue;
            p->split = (int)split;
            p->blocks = rows * split;
            p->min_chunk = 0;
            p->workspace = 0;
            return RMSN_OK;
        }
        p->split = 0;
        // a share is at least two steps for each of its warps; no more shares
        // than the longest rows that the table holds would fill
        p->min_chunk = 2 * warps;
        const int64_t full = (total + p->min_chunk - 1) / p->min_chunk;
        p->blocks = full < resident ? full : resident;
        if (total / p->blocks > (1 << 30)) return RMSN_EUNSUPPORTED;  // a share counts in 31 bits
        // a thread joins eight parts at once; more groups of threads where a
        // row has more
        p->join = p->blocks / rows < 8 ? (int)head_dim : 512;
        p->workspace = p->blocks * (kCutBytes + 2 * (int64_t)e->part * 4);
    }
    return RMSN_OK;
}

void fill_attend(const Plan& p, int64_t n_queries, int64_t n_q_heads, AttendArgs* a) {
    a->n = (int32_t)n_queries;
    a->Hq = (int32_t)n_q_heads;
    a->cols = (int32_t)(n_q_heads / a->c.H * n_queries);
    a->group = (int32_t)(n_q_heads / a->c.H);
    a->group_rcp = ((uint64_t(1) << 32) + a->group - 1) / a->group;
    a->groups = p.groups;
    a->page_rcp = ((uint64_t(1) << 37) + a->c.page / kBlock - 1) / (a->c.page / kBlock);
    a->split = p.split;
    while ((1 << a->split_log) < a->split) ++a->split_log;
    a->shares = p.blocks;
    a->min_chunk = p.min_chunk;
}

int launch_attend(const Plan& p, AttendArgs* a, bool pdl, cudaStream_t stream, int which) {
    const int st = which & 1 ? launch(p.e->fn, dim3((unsigned)p.blocks), p.e->threads, (size_t)p.e->smem, a,
                                      pdl, stream, p.split > 1 ? p.split : 1)
                             : RMSN_OK;
    if (st != RMSN_OK || !(which & 2) || p.split > 0 || p.blocks == 1) return st;
    // always behind the stream's own kernel: a programmatic dependent of it
    const int used = a->cols < 8 * p.e->NT ? a->cols : 8 * p.e->NT;
    return launch(p.e->join, dim3((unsigned)(p.blocks - 1), (unsigned)(used + 3) / 4), p.join, 0, a, true,
                  stream);
}

}  // namespace rmsattn

RMSATTN_API int64_t rmsattn_kv_attention_workspace(int64_t n_seqs, int64_t n_queries,
                                                   int64_t n_q_heads, int64_t n_kv_heads,
                                                   int64_t head_dim, int64_t max_tokens, int64_t window,
                                                   int64_t sinks) {
    const int st = check_attend(n_seqs, n_queries, n_q_heads, n_kv_heads, head_dim);
    if (st != RMSN_OK) return st;
    if (max_tokens < 0 || max_tokens > kMaxTokens || window < 0 || sinks < 0) return RMSN_EINVAL;
    if (n_seqs == 0) return 0;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    Plan p;  // both dtypes' kernels have the same shape
    const int sp = plan_attend(d, false, RMSN_IN_BF16, n_seqs, n_queries, n_q_heads, n_kv_heads, head_dim,
                               max_tokens, window, sinks, &p);
    return sp == RMSN_OK ? p.workspace : sp;
}

RMSATTN_API int rmsattn_kv_attention(const void* q, const rmsattn_cache* cache,
                                     const int32_t* block_table, int64_t table_stride,
                                     int64_t table_width, const int32_t* lengths, void* out,
                                     int64_t q_stride, int64_t out_stride, int64_t n_seqs,
                                     int64_t n_queries, int64_t n_q_heads, float scale,
                                     int64_t window, int64_t sinks, void* workspace,
                                     int64_t workspace_bytes, uint32_t flags,
                                     cudaStream_t stream) {
    if (flags & ~(RMSN_IN_MASK | RMSN_PDL)) return RMSN_EINVAL;
    int64_t bytes = 0;
    const int dt = dtype_of(flags, &bytes);
    if (dt < 0) return RMSN_EINVAL;
    if (dt == RMSN_IN_F32) return RMSN_EUNSUPPORTED;
    AttendArgs a;
    memset(&a, 0, sizeof(a));
    int st = check_cache(cache, &a.c);
    if (st != RMSN_OK) return st;
    st = check_attend(n_seqs, n_queries, n_q_heads, a.c.H, a.c.D);
    if (st != RMSN_OK) return st;
    if (!isfinite(scale) || window < 0 || sinks < 0) return RMSN_EINVAL;
    const int64_t width = n_q_heads * a.c.D;
    if (q_stride < width || out_stride < width || (q_stride * bytes) % 16 ||
        (out_stride * bytes) % 16)
        return RMSN_EINVAL;
    if (too_big(times(n_seqs * n_queries, times(q_stride, 2))) ||
        too_big(times(n_seqs * n_queries, times(out_stride, 2))))
        return RMSN_EINVAL;
    st = check_table(block_table, table_stride, table_width, n_seqs, a.c.page);
    if (st != RMSN_OK) return st;
    if (n_seqs == 0) return RMSN_OK;
    if (!q || !out || !lengths) return RMSN_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(workspace, 16))
        return RMSN_EALIGN;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    Plan p;
    st = plan_attend(d, false, dt, n_seqs, n_queries, n_q_heads, a.c.H, a.c.D, table_width * a.c.page,
                     window, sinks, &p);
    if (st != RMSN_OK) return st;
    if (p.workspace > 0 && (!workspace || workspace_bytes < p.workspace)) return RMSN_EINVAL;
    if (a.c.n_pages == 0) {  // nothing is read; copies of no bytes still name an address
        a.c.k = a.c.v = (uint8_t*)q;
        a.c.ks = a.c.vs = (float*)q;
    }
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.lengths = lengths;
    a.B = n_seqs;
    a.scale = scale;
    // wider than any position: every earlier token
    a.window = window >= kMaxTokens ? 0 : (int32_t)window;
    a.sinks = (int32_t)(sinks > kMaxTokens ? kMaxTokens : sinks);
    a.pdl = (flags & RMSN_PDL) ? 1 : 0;
    a.status = d->status;
    a.ws = static_cast<char*>(workspace);
    fill_attend(p, n_queries, n_q_heads, &a);
    return launch_attend(p, &a, a.pdl, stream);
}

RMSATTN_API int rmsattn_read_status(uint32_t* status, int clear) {
    if (!status) return RMSN_EINVAL;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    if (cudaMemcpy(status, d->status, sizeof(uint32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
        return RMSN_ECUDA;
    if (clear && *status && cudaMemset(d->status, 0, sizeof(uint32_t)) != cudaSuccess)
        return RMSN_ECUDA;
    return RMSN_OK;
}

RMSATTN_API int rmsattn_set_wait_limit(int64_t cycles) {
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    d->wait_cycles.store(cycles == 0 ? kWaitCycles : cycles, std::memory_order_relaxed);
    return RMSN_OK;
}
