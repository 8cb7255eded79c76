// Host helpers that the C-ABI units share: device facts, argument checks, launches
// and the attention's plan.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "../../include/rmsnorm_attn.h"
#include "attn_args.h"

#define RMSATTN_API extern "C" __attribute__((visibility("default")))

namespace rmsattn {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxTokens = int64_t(1) << 29;  // tokens that a table's row may hold

struct DeviceInfo {
    std::once_flag once;
    int num_sms = 0;
    uint32_t* status = nullptr;
    cudaError_t err = cudaSuccess;
    std::atomic<int64_t> wait_cycles{kWaitCycles};  // (tests may lower it)
    std::mutex mu;
    struct {
        const void* fn;
        int64_t blocks;
    } resident[64];  // a kernel's resident blocks, once asked for
    int n_resident = 0;
};

// The current device's, or NULL.
DeviceInfo* device_info();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// RMSN_IN_* of flags, or -1; `bytes`: its element size.
inline int dtype_of(uint32_t flags, int64_t* bytes) {
    const uint32_t in = flags & RMSN_IN_MASK;
    if (in != RMSN_IN_F32 && in != RMSN_IN_BF16 && in != RMSN_IN_F16) return -1;
    *bytes = in == RMSN_IN_F32 ? 4 : 2;
    return (int)in;
}

// a * b without overflow for sizes (>= 0), saturating far above any memory.
inline int64_t times(int64_t a, int64_t b) {
    if (a != 0 && b > (INT64_MAX / 64) / a) return INT64_MAX / 64;
    return a * b;
}
inline bool too_big(int64_t n) { return n >= INT64_MAX / 64; }

int launch(const void* fn, dim3 grid, int threads, size_t smem, void* args, bool pdl,
           cudaStream_t stream, int cluster = 1);

// The cache's shape and pointers; fills the kernels' form of it.
int check_cache(const rmsattn_cache* c, Cache* out);

// Bytes that a call reads or writes: `rows` pieces of `bytes`, `stride` bytes apart.
struct Bytes {
    uintptr_t at;
    uint64_t bytes, rows = 1, stride = 0;
};
inline Bytes bytes_of(const void* p, int64_t n, int64_t rows = 1, int64_t stride = 0) {
    return {reinterpret_cast<uintptr_t>(p), (uint64_t)n, (uint64_t)rows, (uint64_t)stride};
}
// Whether a piece [p, p + n) meets one of r's.
inline bool meets(uintptr_t p, uint64_t n, const Bytes& r) {
    if (n == 0 || r.bytes == 0 || r.rows == 0 || p + n <= r.at) return false;
    const uint64_t from = p > r.at ? p - r.at : 0;  // of the piece, from r's first byte on
    const uint64_t row = r.stride ? from / r.stride : 0;
    if (row < r.rows && from - row * r.stride < r.bytes) return true;
    return row + 1 < r.rows && p + n - r.at > (row + 1) * r.stride;
}

// Block table of n_seqs rows.
int check_table(const int32_t* table, int64_t stride, int64_t width, int64_t n_seqs, int page);

// Sizes of an attention call, before any device is asked.
int check_attend(int64_t n_seqs, int64_t n_queries, int64_t n_q_heads, int64_t n_kv_heads,
                 int64_t head_dim);

// Resident blocks of a kernel on the device (its grid), at most per_sm an SM, or 0.
int64_t resident_blocks(DeviceInfo* d, const void* fn, int threads, int smem, int per_sm);

// How an attention call's steps are shared out.
struct Plan {
    const AttendEntry* e;
    int groups;      // column groups of a key head
    int split;       // a row to `split` blocks of a cluster; 0: one line of all steps
    int64_t blocks;  // of the grid; shares of the line
    int join;        // threads of a block of the join
    int64_t min_chunk;
    int64_t workspace;
};

// `behind`: the kernels that start behind a shared prefix.
int plan_attend(DeviceInfo* d, bool behind, int dt, int64_t n_seqs, int64_t n_queries,
                int64_t n_q_heads, int64_t n_kv_heads, int64_t head_dim, int64_t max_tokens,
                int64_t window, int64_t sinks, Plan* p);

// The attention's and its join's launches, once every pointer is in `a`.
void fill_attend(const Plan& p, int64_t n_queries, int64_t n_q_heads, AttendArgs* a);
// (which: 1 the attention alone, 2 its join, 3 both)
int launch_attend(const Plan& p, AttendArgs* a, bool pdl, cudaStream_t stream, int which = 3);

}  // namespace rmsattn
