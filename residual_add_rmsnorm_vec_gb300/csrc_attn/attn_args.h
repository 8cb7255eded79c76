// Kernel arguments and tables of the attention-path operators, shared by the
// kernels' units and the C-ABI layer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsattn {

constexpr int kBlock = 16;          // tokens that share a cache scale
constexpr uint32_t kBadPage = 4u;   // status bit: a page or token outside the cache
constexpr uint32_t kWaitRanOut = 1u;  // status bit: a kernel gave up a wait
constexpr long long kWaitCycles = 2000000000LL;  // before it does: about a second

// q / k: first element of token 0's first head; strides in elements.
struct RopeArgs {
    const void* q;
    const void* k;
    const void* qw;
    const void* kw;
    void* qo;
    void* ko;
    const void* pos;
    const uint64_t* turns;
    const int32_t* axis;
    int64_t T, pos_stride, qs, ks, qos, kos;
    int32_t Hq, Hk, D, R;
    int32_t n_axes;
    int32_t norm, interleaved, pos64, pdl;
    float eps, woff;
    float rcp_d;  // 1 / head_dim when that is exact, else 0
};

constexpr int kRopeWarps = 8;  // of a block, at most

// One compiled 16-byte-vector rotary kernel: tph lanes a head, u tokens a block.
struct RopeEntry {
    int32_t dt, tph, u, interleaved;
    const void* fn;
};
const RopeEntry* rope_kernels(int* n);

struct Cache {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int64_t n_pages, page_stride, scale_stride;
    int32_t H, page, D;
};

struct AppendArgs {
    Cache c;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;
    const int32_t* table;
    int64_t table_stride, table_width;
    const int32_t* lengths;
    const int32_t* cu;  // NULL: one token per sequence
    int64_t T, B;
    int32_t pdl;
    uint32_t* status;
};

// A serving step's plan; `more`: the tokens that each sequence gets (negative:
// it is finished).
struct PagesArgs {
    int32_t* free_pages;
    const int32_t* n_free;
    int32_t* table;
    int64_t table_stride, width, n_pages;
    const int32_t* lengths;
    const int32_t* more;
    const int32_t* shared;  // pages of a row that are not the sequence's own, or NULL
    int64_t B, T;
    int32_t page, pdl;
    int32_t *cu, *positions, *rows, *before, *after, *n_free_out;
    int64_t* slots;
    int32_t* ws;
    uint32_t* status;
};
constexpr int64_t kPagesOnce = 2048;  // sequences that one launch takes
// 0: one launch; 1, 2: the scan and the rows
const void* pages_kernel_of(int which);

// The norms at a block's end; gate_stride 0: one row for all.
struct NormsArgs {
    const void *x, *residual, *post_w, *w, *gate;
    const int32_t* index;  // a row's gate row; negative: the row is left out
    void *out, *residual_out;
    float* out_scale;
    int64_t T, gate_stride, n_gates;
    int32_t H, pdl;
    float eps, alpha, w_off;
    bool zero_out, zero_residual, zero_scale;  // of a row that is left out (else as it was)
    uint32_t* status;
};
// ch vectors of eight elements to a thread; 0: any row
const void* norms_kernel_of(int dt, bool r32, bool fp8, bool ragged, int ch);

// A group of sequences [s0, s1) that share their first `shared` tokens: `tiles`
// tiles of `rows` columns (sequence x query token x head) for each key head,
// an item each; an item is ns steps, the group's items lie one behind the other
// on the line of all steps from `first` on.  Their parts' rows, in eights and for
// all key heads, are counted from row0 on.
struct __align__(16) PrefixGroup {
    int32_t s0, s1, shared;
    int32_t seq;  // the sequence whose table row names the shared pages
    int32_t ns, first, row0, tiles;
};
// The line of the shared parts: total steps, and the steps of a share.
struct __align__(16) PrefixLine {
    int32_t total, chunk, pad[2];
};
// A sequence's shared tokens (0: it does not share) and its group.
struct PrefixSeq {
    int32_t start, group;
};

struct PrefixArgs {
    Cache c;
    const void* q;
    int64_t q_stride;
    const int32_t* table;
    int64_t table_stride, table_width;
    const int32_t* lengths;
    const int32_t* cu;      // borders of the groups, or NULL: one group of all
    const int32_t* shared;  // tokens that each group shares
    int64_t B;
    int32_t n_groups, n, group;  // group: query heads of a key head
    int32_t tok, rows;           // tokens of a step, columns of an item
    int32_t shares;
    int32_t pdl;
    float scale;
    uint64_t page_rcp;  // ceil(2^37 / (page / 16))
    long long wait_cycles;  // of each wait inside a block, at most
    uint32_t* status;
    PrefixLine* line;
    PrefixGroup* groups;
    PrefixSeq* seqs;
    float* parts;  // one for each pair of a share and an item that it meets
};
// A part's rows stand in eights: their sums [D / 8][8][8], then reference and weight of each,
// 8 (D + 2) floats.  A group has its columns' eights for each key head, most / 8 in each of its
// tiles but the last, so that small groups take no whole tiles.  Share s's part of an item whose
// rows begin at eight e begins at eight s most / 8 + e: behind the share's part of the item
// before, and behind the earlier share's part of the same item.  (Columns are counted in 31
// bits, and so are the eights.)
__host__ __device__ constexpr uint32_t prefix_eights(uint32_t columns) { return (columns + 7) / 8; }
// First eight of an item.
__host__ __device__ constexpr uint32_t prefix_eight(const PrefixGroup& g, int per_seq, int hk, int tile, int most) {
    return g.row0 + hk * prefix_eights((uint32_t)(g.s1 - g.s0) * per_seq) + tile * (most / 8);
}

// One compiled kernel: R tiles of 128 rows.
struct PrefixEntry {
    int32_t dt, D, R, tok, threads, smem;
    const void* fn;
};
const void* prefix_plan_kernel();

// The join of a sequence's own part with its group's.
struct PrefixJoinArgs {
    void* out;
    int64_t out_stride, rows;  // rows: B n Hq
    int32_t n, Hq, group, D;
    int32_t item_rows;
    const PrefixLine* line;
    const PrefixGroup* groups;
    const PrefixSeq* seqs;
    const float* parts;
    const float* own;
    const float2* own_ml;
};
const void* prefix_join_kernel(int dt, int ways);  // 1 or 4
const PrefixEntry* prefix_kernels_64(int* n);
const PrefixEntry* prefix_kernels_128(int* n);
const PrefixEntry* prefix_kernels_256(int* n);

struct AttendArgs {
    Cache c;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    const int32_t* table;
    int64_t table_stride, table_width;
    const int32_t* lengths;
    int64_t B;
    int32_t n, Hq;
    float scale;
    int32_t window, sinks;  // window 0: every earlier token
    int32_t pdl;
    uint32_t* status;
    // how the steps are shared out: 0, as one line; else a row to `split` blocks
    int32_t split, split_log;  // a power of two
    int32_t groups;     // column groups of a key head
    int32_t cols;       // columns of a key head: query heads x query tokens
    int32_t group;      // query heads of a key head
    uint64_t group_rcp; // ceil(2^32 / group): exact quotients of up to 2^17 columns
    uint64_t page_rcp;  // ceil(2^37 / (page / 16))
    int64_t shares;     // of the line, one for each block
    int64_t min_chunk;  // steps of a share, at least
    char* ws;           // a Cut and two parts for every share
    // behind a shared prefix: where each sequence begins, and its own tokens' results
    // [B, n, Hq, D] with each row's reference and weight
    const PrefixSeq* seqs;
    float* own;
    float2* own_ml;
};

constexpr int64_t kCutBytes = 32;
constexpr int kMaxSplit = 8;  // blocks of a cluster

// One compiled attention kernel and the join of its parts.
struct AttendEntry {
    int32_t dt, D, NT, tok, threads, smem;
    int32_t per_sm;  // blocks an SM holds: the same for every dtype of a shape
    int32_t most;  // takes rows of up to this many tokens
    int32_t part;  // floats of one part
    const void* fn;
    const void* join;
};
const AttendEntry* attend_kernels_64(int* n);
const AttendEntry* attend_kernels_128(int* n);
const AttendEntry* attend_kernels_256(int* n);
// the same for sequences that begin behind a shared prefix
const AttendEntry* attend_behind_64(int* n);
const AttendEntry* attend_behind_128(int* n);
const AttendEntry* attend_behind_256(int* n);

// dt: 0 fp32, 1 bf16, 2 fp16 (the RMSN_IN_* values)
const void* rope_generic_kernel(int dt);
const void* append_kernel_of(int dt, int D, bool vec);

}  // namespace rmsattn
