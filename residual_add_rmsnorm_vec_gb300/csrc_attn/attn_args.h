// Kernel arguments and tables of the attention-path operators, shared by the
// kernels' units and the C-ABI layer.
#pragma once

#include <stdint.h>

namespace rmsattn {

constexpr int kBlock = 16;          // tokens that share a cache scale
constexpr uint32_t kBadPage = 4u;   // status bit: a page or token outside the cache

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

// dt: 0 fp32, 1 bf16, 2 fp16 (the RMSN_IN_* values)
const void* rope_generic_kernel(int dt);
const void* append_kernel_of(int dt, int D, bool vec);

}  // namespace rmsattn
