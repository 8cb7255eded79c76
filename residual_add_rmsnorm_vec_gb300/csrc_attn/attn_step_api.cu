// C ABI of the operators around the attention in a serving step: the page plan,
// attention with a shared prefix, the norms at a block's end.
#include <math.h>
#include <string.h>

#include "attn_host.h"

using namespace rmsattn;

// ---------------------------------------------------------------- pages

RMSATTN_API int64_t rmsattn_pages_workspace(int64_t n_seqs) {
    if (n_seqs < 0 || n_seqs > (1 << 24)) return RMSN_EINVAL;
    return n_seqs <= kPagesOnce ? 0 : (4 + 3 * (n_seqs + 1)) * 4;
}

RMSATTN_API int rmsattn_pages_step(int32_t* free_pages, int64_t n_pages, const int32_t* n_free,
                                   int32_t* block_table, int64_t table_stride, int64_t table_width,
                                   const int32_t* lengths, const int32_t* new_tokens,
                                   const int32_t* shared_pages, int64_t n_seqs, int64_t page_size,
                                   int64_t n_rows, int32_t* cu_seqlens, int32_t* positions,
                                   int64_t* slots, int32_t* rows, int32_t* before, int32_t* after,
                                   int32_t* n_free_out, void* workspace, int64_t workspace_bytes,
                                   uint32_t flags, cudaStream_t stream) {
    if (flags & ~RMSN_PDL) return RMSN_EINVAL;
    if (n_pages < 0 || n_pages > INT32_MAX || n_seqs < 0 || n_seqs > (1 << 24) || n_rows < 0 ||
        n_rows > kMaxTokens || page_size < kBlock || page_size > 65536 || page_size % kBlock)
        return RMSN_EINVAL;
    const int st = check_table(block_table, table_stride, table_width, n_seqs, (int)page_size);
    if (st != RMSN_OK) return st;
    if (!n_free || !cu_seqlens || !n_free_out || (n_pages && !free_pages)) return RMSN_EINVAL;
    if (n_seqs && (!lengths || !new_tokens || !before || !after)) return RMSN_EINVAL;
    if (n_rows && (!positions || !slots || !rows)) return RMSN_EINVAL;
    const void* words[] = {free_pages, n_free, lengths, new_tokens, shared_pages, cu_seqlens,
                           before,     after,  n_free_out};
    for (const void* p : words)
        if (!aligned(p, 4)) return RMSN_EALIGN;
    if (!aligned(positions, 16) || !aligned(slots, 16) || !aligned(rows, 16) || !aligned(workspace, 16))
        return RMSN_EALIGN;
    const int64_t need = rmsattn_pages_workspace(n_seqs);
    if (need && (!workspace || workspace_bytes < need)) return RMSN_EINVAL;
    // Blocks read the inputs while others write: what is written lies apart from all else.
    const Bytes written[] = {bytes_of(cu_seqlens, (n_seqs + 1) * 4), bytes_of(positions, n_rows * 4),
                             bytes_of(slots, n_rows * 8), bytes_of(rows, n_rows * 4),
                             bytes_of(before, n_seqs * 4), bytes_of(after, n_seqs * 4),
                             bytes_of(n_free_out, 4), bytes_of(workspace, need), bytes_of(free_pages, n_pages * 4)};
    const Bytes read[] = {bytes_of(block_table, table_width * 4, n_seqs, table_stride * 4),
                          bytes_of(n_free, 4), bytes_of(lengths, n_seqs * 4), bytes_of(new_tokens, n_seqs * 4),
                          bytes_of(shared_pages, shared_pages ? n_seqs * 4 : 0)};
    constexpr int kWritten = sizeof(written) / sizeof(written[0]);
    for (int i = 0; i < kWritten; ++i) {
        for (int k = 0; k < i; ++k)
            if (meets(written[i].at, written[i].bytes, written[k])) return RMSN_EINVAL;
        for (const Bytes& r : read)
            if (meets(written[i].at, written[i].bytes, r)) return RMSN_EINVAL;
    }
    for (const Bytes& r : read)  // (the table is written, too)
        if (&r != read && meets(r.at, r.bytes, read[0])) return RMSN_EINVAL;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    PagesArgs a;
    memset(&a, 0, sizeof(a));
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.table = block_table;
    a.table_stride = table_stride;
    a.width = table_width;
    a.n_pages = n_pages;
    a.lengths = lengths;
    a.more = new_tokens;
    a.shared = shared_pages;
    a.B = n_seqs;
    a.T = n_rows;
    a.page = (int32_t)page_size;
    a.pdl = (flags & RMSN_PDL) ? 1 : 0;
    a.cu = cu_seqlens;
    a.positions = positions;
    a.rows = rows;
    a.before = before;
    a.after = after;
    a.n_free_out = n_free_out;
    a.slots = slots;
    a.ws = static_cast<int32_t*>(workspace);
    a.status = d->status;
    // Up to four rows to a thread; a warp to a sequence (one that returns pages has a row of
    // them to read: with 32 sequences to a warp, 1024 x 1 token took 2.3 times as long).  Small
    // blocks while their scan of all sequences is short and there are SMs for them: 8 x 1 token
    // take 0.87 of the large ones' time, 64 x 200 0.89, but 1024 x 1 1.14, 64 x 2000 1.04.
    const int threads = n_seqs <= 256 && n_rows <= 512 * (int64_t)d->num_sms ? 128 : 512;
    int64_t blocks = (n_rows + 4 * threads - 1) / (4 * threads);
    const int64_t by_seqs = (n_seqs * 32 + threads - 1) / threads;
    if (blocks < by_seqs) blocks = by_seqs;
    if (blocks > d->num_sms) blocks = d->num_sms;
    if (blocks < 1) blocks = 1;
    if (n_seqs <= kPagesOnce)
        return launch(pages_kernel_of(0), dim3((unsigned)blocks), threads, (size_t)(3 * (n_seqs + 1)) * 4, &a,
                      a.pdl, stream);
    const int sc = launch(pages_kernel_of(1), dim3(1), 1024, 0, &a, a.pdl, stream);
    return sc != RMSN_OK ? sc : launch(pages_kernel_of(2), dim3((unsigned)blocks), threads, 0, &a, true, stream);
}

// ---------------------------------------------------------------- norms

RMSATTN_API int rmsattn_block_norms(const void* x, const void* residual, const void* post_weight,
                                    const void* weight, const void* gate, int64_t gate_stride,
                                    const int32_t* gate_index, int64_t n_gates, void* out,
                                    void* residual_out, float* out_scale, int64_t n_tokens,
                                    int64_t hidden, float eps, float residual_scale, float weight_offset,
                                    uint32_t flags, cudaStream_t stream) {
    if (flags & ~(RMSN_IN_MASK | RMSN_RESIDUAL_F32 | RMSATTN_OUT_FP8 | RMSN_PDL | RMSATTN_ZERO_OUT |
                  RMSATTN_ZERO_RESIDUAL | RMSATTN_ZERO_SCALE))
        return RMSN_EINVAL;
    int64_t bytes = 0;
    const int dt = dtype_of(flags, &bytes);
    if (dt < 0) return RMSN_EINVAL;
    const bool r32 = (flags & RMSN_RESIDUAL_F32) != 0, fp8 = (flags & RMSATTN_OUT_FP8) != 0;
    if (r32 && dt == RMSN_IN_F32) return RMSN_EINVAL;
    if (n_tokens < 0 || n_tokens > INT32_MAX || hidden < 1 || hidden > (1 << 24)) return RMSN_EINVAL;
    if (too_big(times(n_tokens, hidden * 4))) return RMSN_EINVAL;
    if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(residual_scale) || !isfinite(weight_offset))
        return RMSN_EINVAL;
    if (gate_stride < 0 || (gate_stride > 0 && gate_stride < hidden) || n_gates < 0 ||
        too_big(times(n_gates, times(gate_stride, 4))))
        return RMSN_EINVAL;
    if (fp8 ? (n_tokens && !out_scale) : out_scale != nullptr) return RMSN_EINVAL;
    if (!fp8 && (flags & RMSATTN_ZERO_SCALE)) return RMSN_EINVAL;
    if (n_tokens == 0) return RMSN_OK;
    // From here on the pointers say what the gate is.  (An empty tensor's may be NULL: without
    // tokens those of the index and of each token's gate, and of gates that are none at all,
    // to which no index leads.)
    if (!gate && (n_gates != 0 || (gate_stride != 0) != (gate_index != nullptr))) return RMSN_EINVAL;
    if (gate_index ? n_gates > INT32_MAX : gate && n_gates != (gate_stride ? n_tokens : 1)) return RMSN_EINVAL;
    if (!x || !residual || !out || !residual_out) return RMSN_EINVAL;
    const int64_t rbytes = r32 ? 4 : bytes;
    const void* same[] = {x, post_weight, weight, gate};
    for (const void* p : same)
        if (!aligned(p, (uintptr_t)bytes)) return RMSN_EALIGN;
    if (!aligned(residual, (uintptr_t)rbytes) || !aligned(residual_out, (uintptr_t)rbytes) ||
        !aligned(out, fp8 ? 1 : (uintptr_t)bytes) || !aligned(out_scale, 4) || !aligned(gate_index, 4))
        return RMSN_EALIGN;
    // A block reads its row before it writes it, so an output may lie on an input row for
    // row; else a block would write what another one reads.
    const int64_t row = hidden * (fp8 ? 1 : bytes), row_r = hidden * rbytes, row_x = hidden * bytes;
    const Bytes outs[] = {bytes_of(out, n_tokens * row), bytes_of(residual_out, n_tokens * row_r),
                          bytes_of(out_scale, fp8 ? n_tokens * 4 : 0)};
    const int64_t out_rows[] = {row, row_r, 0};
    const struct {
        Bytes b;
        int64_t row;  // bytes from row to row, 0: not a row for each token
    } ins[] = {{bytes_of(x, n_tokens * row_x), row_x},
               {bytes_of(residual, n_tokens * row_r), row_r},
               {bytes_of(gate, gate ? row_x : 0, n_gates, gate_stride * bytes), gate_index ? 0 : gate_stride * bytes},
               {bytes_of(post_weight, post_weight ? row_x : 0), 0},
               {bytes_of(weight, weight ? row_x : 0), 0},
               {bytes_of(gate_index, gate_index ? n_tokens * 4 : 0), 0}};
    for (int i = 0; i < 3; ++i) {
        for (int k = 0; k < i; ++k)
            if (meets(outs[i].at, outs[i].bytes, outs[k])) return RMSN_EINVAL;
        for (const auto& in : ins)
            if ((in.b.at != outs[i].at || in.row == 0 || in.row != out_rows[i]) &&
                meets(outs[i].at, outs[i].bytes, in.b))
                return RMSN_EINVAL;
    }
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    NormsArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x;
    a.residual = residual;
    a.post_w = post_weight;
    a.w = weight;
    a.gate = gate;
    a.index = gate_index;
    a.out = out;
    a.residual_out = residual_out;
    a.out_scale = out_scale;
    a.T = n_tokens;
    a.gate_stride = gate_stride;
    a.n_gates = n_gates;
    a.H = (int32_t)hidden;
    a.pdl = (flags & RMSN_PDL) ? 1 : 0;
    a.eps = eps;
    a.alpha = residual_scale;
    a.w_off = weight_offset;
    a.zero_out = (flags & RMSATTN_ZERO_OUT) != 0;
    a.zero_residual = (flags & RMSATTN_ZERO_RESIDUAL) != 0;
    a.zero_scale = (flags & RMSATTN_ZERO_SCALE) != 0;
    a.status = d->status;
    // Vectors of eight elements where the tensors of rows begin on one; where every row,
    // and the weights' and gates', does too, no row has ends of its own.
    bool vec = aligned(out, fp8 ? 8 : (uintptr_t)(8 * bytes)) && aligned(x, (uintptr_t)(8 * bytes)) &&
               aligned(residual, (uintptr_t)(8 * rbytes)) && aligned(residual_out, (uintptr_t)(8 * rbytes));
    bool ragged = hidden % 8 != 0 || gate_stride % 8 != 0;
    for (const void* p : same) ragged = ragged || !aligned(p, (uintptr_t)(8 * bytes));
    // Vectors of a thread: as few as put all rows on the SMs at once, for the shorter chain
    // (8 x 4096 bf16 take 0.9 of the time with one as with four, 900 x 1024 0.82); four
    // otherwise, which put the most rows on an SM (600 x 4096 take 0.84 of the time with four
    // as with one, 2000 x 4096 0.61, 16384 x 8192 0.8 of the time with two).
    const int64_t vectors = (hidden + (ragged ? 14 : 7)) / 8;
    int64_t ch = 1;
    while (ch < 4 && ((vectors + ch - 1) / ch > 512 || n_tokens * ((vectors + ch - 1) / ch) > 1024 * (int64_t)d->num_sms))
        ch *= 2;
    // three where that takes fewer turns of a warp (4099 x 2045: 3 x 86 lanes, or 4 x 65)
    auto turns = [&](int64_t c) { return ((vectors + c - 1) / c + 31) / 32 * c; };
    if (ch == 4 && (vectors + 2) / 3 <= 512 && turns(3) < turns(4)) ch = 3;
    int64_t lanes = (vectors + ch - 1) / ch;
    if (!vec || lanes > 512) {
        ch = 0;
        lanes = hidden < 1024 ? hidden : 1024;
    }
    const int threads = (int)((lanes + 31) / 32 * 32);
    return launch(norms_kernel_of(dt, r32, fp8, ragged, (int)ch), dim3((unsigned)n_tokens), threads, 0, &a, a.pdl, stream);
}

// ---------------------------------------------------------------- shared prefix

namespace {

// Two row tiles where the groups have more than 128 columns on average: they share the
// widening of each key and value (4 heads x 128 to a key head, 300 own tokens: 256 sequences x 8192 tokens 116 against
// 123 us with one; 33 sequences 44 against 46).  One otherwise (32 sequences 40 against 42,
// 8 groups of 32 sequences x 4096 99 against 101).
const PrefixEntry* prefix_entry_of(int dt, int64_t D, int64_t cols, int64_t n_groups) {
    int n = 0;
    const PrefixEntry* t = D == 64 ? prefix_kernels_64(&n)
                                   : (D == 128 ? prefix_kernels_128(&n) : prefix_kernels_256(&n));
    const PrefixEntry* best = nullptr;
    for (int i = 0; i < n; ++i)
        if (t[i].dt == dt && (!best || cols > 128 * (n_groups < 1 ? 1 : n_groups))) best = &t[i];
    return best;
}

// Where a call's workspace holds what.
struct PrefixPlan {
    const PrefixEntry* e;
    int64_t shares, groups, seqs, parts, own, own_ml, behind_ws, total;  // offsets in bytes
    Plan behind;
};

int64_t round_up(int64_t n) { return (n + 255) / 256 * 256; }

int plan_prefix(DeviceInfo* d, int dt, int64_t n_seqs, int64_t n_queries, int64_t n_q_heads,
                int64_t n_kv_heads, int64_t head_dim, int64_t max_tokens, int64_t n_groups, PrefixPlan* p) {
    const int64_t cols = n_seqs * n_queries * (n_q_heads / n_kv_heads);
    p->e = prefix_entry_of(dt, head_dim, cols, n_groups);
    p->shares = resident_blocks(d, p->e->fn, p->e->threads, p->e->smem, 1);
    if (p->shares < 1) return RMSN_ECUDA;
    const int rows = 128 * p->e->R;
    // a group of two sequences or more shares: its columns fill whole tiles but for one
    const int64_t some = n_groups < n_seqs / 2 ? n_groups : n_seqs / 2;
    const int64_t tiles = cols / rows + some;
    const int64_t items = times(tiles, n_kv_heads);
    if (times(items, (max_tokens + p->e->tok - 1) / p->e->tok) + p->shares >= (int64_t(1) << 31))
        return RMSN_EUNSUPPORTED;  // steps are counted in 31 bits
    const int64_t part_rows = times(cols + 7 * some, n_kv_heads);
    if (part_rows / 8 >= (int64_t(1) << 31)) return RMSN_EUNSUPPORTED;  // and eights of rows
    const int st = plan_attend(d, true, dt, n_seqs, n_queries, n_q_heads, n_kv_heads, head_dim, max_tokens,
                               0, 0, &p->behind);
    if (st != RMSN_OK) return st;
    p->groups = round_up(sizeof(PrefixLine));
    p->seqs = p->groups + round_up((n_groups + 1) * (int64_t)sizeof(PrefixGroup));
    p->parts = p->seqs + round_up(n_seqs * (int64_t)sizeof(PrefixSeq));
    p->own = p->parts + round_up(times(p->shares * rows + part_rows, (head_dim + 2) * 4));
    const int64_t out_rows = n_seqs * n_queries * n_q_heads;
    p->own_ml = p->own + times(out_rows, head_dim * 4);
    p->behind_ws = p->own_ml + round_up(out_rows * 8);
    p->total = p->behind_ws + p->behind.workspace;
    return too_big(p->total) ? RMSN_EUNSUPPORTED : RMSN_OK;
}

int check_prefix(int64_t n_seqs, int64_t n_queries, int64_t n_q_heads, int64_t n_kv_heads,
                 int64_t head_dim, int64_t n_groups) {
    if (n_groups < 0 || n_groups > (1 << 24)) return RMSN_EINVAL;
    const int st = check_attend(n_seqs, n_queries, n_q_heads, n_kv_heads, head_dim);
    if (st != RMSN_OK) return st;
    // columns are counted in 31 bits; the join's grid
    if (times(n_seqs * n_queries, n_q_heads / n_kv_heads) >= (int64_t(1) << 31)) return RMSN_EUNSUPPORTED;
    return n_kv_heads * (head_dim / 8) > 65535 ? RMSN_EUNSUPPORTED : RMSN_OK;
}

}  // namespace

RMSATTN_API int64_t rmsattn_kv_prefix_attention_workspace(int64_t n_seqs, int64_t n_queries,
                                                          int64_t n_q_heads, int64_t n_kv_heads,
                                                          int64_t head_dim, int64_t max_tokens,
                                                          int64_t n_groups) {
    const int st = check_prefix(n_seqs, n_queries, n_q_heads, n_kv_heads, head_dim, n_groups);
    if (st != RMSN_OK) return st;
    if (max_tokens < 0 || max_tokens > kMaxTokens) return RMSN_EINVAL;
    if (n_seqs == 0) return 0;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    PrefixPlan p;  // both dtypes' kernels have the same shape
    const int sp = plan_prefix(d, RMSN_IN_BF16, n_seqs, n_queries, n_q_heads, n_kv_heads, head_dim, max_tokens,
                               n_groups, &p);
    return sp == RMSN_OK ? p.total : sp;
}

RMSATTN_API int rmsattn_kv_prefix_attention(const void* q, const rmsattn_cache* cache,
                                            const int32_t* block_table, int64_t table_stride,
                                            int64_t table_width, const int32_t* lengths,
                                            const int32_t* prefix_lengths, const int32_t* group_cu,
                                            int64_t n_groups, void* out, int64_t q_stride,
                                            int64_t out_stride, int64_t n_seqs, int64_t n_queries,
                                            int64_t n_q_heads, float scale, void* workspace,
                                            int64_t workspace_bytes, uint32_t flags, cudaStream_t stream) {
    if (flags & ~(RMSN_IN_MASK | RMSN_PDL)) return RMSN_EINVAL;
    int64_t bytes = 0;
    const int dt = dtype_of(flags, &bytes);
    if (dt < 0) return RMSN_EINVAL;
    if (dt == RMSN_IN_F32) return RMSN_EUNSUPPORTED;
    AttendArgs a;
    memset(&a, 0, sizeof(a));
    int st = check_cache(cache, &a.c);
    if (st != RMSN_OK) return st;
    st = check_prefix(n_seqs, n_queries, n_q_heads, a.c.H, a.c.D, n_groups);
    if (st != RMSN_OK) return st;
    if (!isfinite(scale)) return RMSN_EINVAL;
    const int64_t width = n_q_heads * a.c.D;
    if (q_stride < width || out_stride < width || (q_stride * bytes) % 16 || (out_stride * bytes) % 16)
        return RMSN_EINVAL;
    if (too_big(times(n_seqs * n_queries, times(q_stride, 2))) ||
        too_big(times(n_seqs * n_queries, times(out_stride, 2))))
        return RMSN_EINVAL;
    st = check_table(block_table, table_stride, table_width, n_seqs, a.c.page);
    if (st != RMSN_OK) return st;
    if (!group_cu && n_groups > 1) return RMSN_EINVAL;
    if (n_seqs == 0) return RMSN_OK;
    if (!q || !out || !lengths || (n_groups && !prefix_lengths) || !workspace) return RMSN_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(workspace, 32) ||
        !aligned(prefix_lengths, 4) || !aligned(group_cu, 4))
        return RMSN_EALIGN;
    DeviceInfo* d = device_info();
    if (!d) return RMSN_ECUDA;
    PrefixPlan p;
    st = plan_prefix(d, dt, n_seqs, n_queries, n_q_heads, a.c.H, a.c.D, table_width * a.c.page, n_groups, &p);
    if (st != RMSN_OK) return st;
    if (workspace_bytes < p.total) return RMSN_EINVAL;
    if (a.c.n_pages == 0) {  // nothing is read; copies of no bytes still name an address
        a.c.k = a.c.v = (uint8_t*)q;
        a.c.ks = a.c.vs = (float*)q;
    }
    char* ws = static_cast<char*>(workspace);
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
    a.status = d->status;
    a.pdl = 1;
    a.ws = ws + p.behind_ws;
    fill_attend(p.behind, n_queries, n_q_heads, &a);

    PrefixArgs f;
    memset(&f, 0, sizeof(f));
    f.c = a.c;
    f.q = q;
    f.q_stride = q_stride;
    f.table = block_table;
    f.table_stride = table_stride;
    f.table_width = table_width;
    f.lengths = lengths;
    f.cu = group_cu;
    f.shared = prefix_lengths;
    f.B = n_seqs;
    f.n_groups = (int32_t)n_groups;
    f.n = (int32_t)n_queries;
    f.group = a.group;
    f.tok = p.e->tok;
    f.rows = 128 * p.e->R;
    f.shares = (int32_t)p.shares;
    f.pdl = (flags & RMSN_PDL) ? 1 : 0;
    f.scale = scale;
    f.page_rcp = a.page_rcp;
    f.wait_cycles = d->wait_cycles.load(std::memory_order_relaxed);
    f.status = d->status;
    f.line = reinterpret_cast<PrefixLine*>(ws);
    f.groups = reinterpret_cast<PrefixGroup*>(ws + p.groups);
    f.seqs = reinterpret_cast<PrefixSeq*>(ws + p.seqs);
    f.parts = reinterpret_cast<float*>(ws + p.parts);
    a.seqs = f.seqs;
    a.own = reinterpret_cast<float*>(ws + p.own);
    a.own_ml = reinterpret_cast<float2*>(ws + p.own_ml);
    PrefixJoinArgs j;
    memset(&j, 0, sizeof(j));
    j.out = out;
    j.out_stride = out_stride;
    j.rows = n_seqs * n_queries * n_q_heads;
    j.n = (int32_t)n_queries;
    j.Hq = (int32_t)n_q_heads;
    j.group = a.group;
    j.D = a.c.D;
    j.item_rows = f.rows;
    j.line = f.line;
    j.groups = f.groups;
    j.seqs = f.seqs;
    j.parts = f.parts;
    j.own = a.own;
    j.own_ml = a.own_ml;
    // Each launch is a programmatic dependent of the one before.  The shared part needs the
    // plan alone, not the own tokens' kernel: it starts beside that one, on the SMs that it
    // leaves or does not take, and waits for it in the end, so that what comes behind finds
    // both done.
    st = launch(prefix_plan_kernel(), dim3(1), 512, 0, &f, f.pdl, stream);
    if (st == RMSN_OK) st = launch_attend(p.behind, &a, true, stream, 1);
    if (st == RMSN_OK && n_groups)
        st = launch(p.e->fn, dim3((unsigned)p.shares), p.e->threads, (size_t)p.e->smem, &f, true, stream);
    if (st == RMSN_OK) st = launch_attend(p.behind, &a, true, stream, 2);
    if (st != RMSN_OK) return st;
    // Four threads to a row's parts where an item has many, for there are few items: the call of
    // 8 sequences x 2048 tokens takes 0.88 of the time so, 64 x 8192 0.92; one else: with four
    // 256 x 8192 take 1.03 of the time, 512 x 4096 1.05.
    const int64_t cols = n_seqs * n_queries * a.group, items = (cols + f.rows - 1) / f.rows * a.c.H;
    const int ways = items * 8 >= p.shares ? 1 : 4;
    return launch(prefix_join_kernel(dt, ways), dim3((unsigned)((cols * ways + 255) / 256), (unsigned)(a.c.H * (a.c.D / 8))),
                  256, 0, &j, true, stream);
}
