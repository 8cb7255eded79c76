/*
 * rmsnorm_attn.h -- C ABI of the GB300 (sm_103a) attention-path operators
 * that stand next to the QK norm of rmsnorm.h: rotary positions with several
 * axes fused with that norm, the append of keys and values to a paged 8-bit
 * cache, and the attention that reads it.  Built into a library of its own
 * (librmsnorm_attn_gb300.so); statuses, dtype flags and RMSN_PDL are those of
 * rmsnorm.h.
 *
 * Ownership: every buffer belongs to the caller, workspaces included; the
 * library allocates no device memory and keeps per-device attributes only.
 * All calls are asynchronous on `stream` (NULL = the legacy default stream),
 * run on the current device, may be captured into a CUDA graph, and are
 * thread-safe.  Argument errors are returned before anything is launched; a
 * launch failure returns RMSN_ECUDA.  Inference only: nothing here has a
 * backward pass.
 */
#ifndef RMSNORM_ATTN_GB300_H
#define RMSNORM_ATTN_GB300_H

#include "rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* flags of rmsattn_qk_rope_fwd (with RMSN_IN_* and RMSN_PDL) */
#define RMSATTN_NORM 0x1000u        /* RMS norm of each head before the rotation */
#define RMSATTN_INTERLEAVED 0x2000u /* pairs are neighbours (2p, 2p + 1) */
#define RMSATTN_POS_I64 0x4000u     /* positions are int64 (else int32) */

/*
 * QK norm and rotary positions of query and key heads in one launch.  Per
 * head x of head_dim elements of token t:
 *
 *   y = (w + weight_offset) * (x * rsqrt(sum(x^2) / head_dim + eps))   with RMSATTN_NORM
 *   y = x                                                             without
 *   for each pair p < rot_dim / 2, elements (i, j) = (p, p + rot_dim / 2), or
 *   (2p, 2p + 1) with RMSATTN_INTERLEAVED:
 *     a = 2 pi * frac(positions[axis[p]][t] * turns[p] / 2^64)
 *     out_i = y_i cos a - y_j sin a;   out_j = y_j cos a + y_i sin a
 *   out_e = y_e for e >= rot_dim
 *
 * in fp32, rounded once to the element type.  turns[p] is the pair's
 * frequency in turns per position as a 64-bit fixed-point fraction,
 * round(inv_freq[p] / (2 pi) * 2^64) mod 2^64: the product with an integer
 * position wraps exactly as the angle does, so far and negative positions
 * lose nothing (the phase is off by |position| * 2^-65 turns at most, the
 * rounding of turns[p], plus fp32's rounding of one turn).  axis[p] < n_axes
 * names the axis (time, height, width, ...) whose position turns the pair.
 *
 *   q, k            [n_tokens, heads, head_dim], token strides in elements
 *   q_out, k_out    the same; q_out may be q (and k_out k) at the same stride;
 *                   any other overlap is undefined
 *   q_weight, k_weight [head_dim] or NULL (1); only read with RMSATTN_NORM
 *   positions       [n_axes, n_tokens] int32 or int64, rows pos_stride apart
 *                   (0: every axis reads the same row)
 *   turns, axis     [rot_dim / 2] on the device
 *
 * rot_dim is even and at most head_dim (0: no rotation); head_dim <= 4096.
 * Any strides and alignments of whole elements run; 16-byte vectors are used
 * where pointers, strides and head_dim allow it.  n_tokens == 0 is a no-op.
 */
int rmsattn_qk_rope_fwd(const void* q, const void* k, const void* q_weight, const void* k_weight,
                        void* q_out, void* k_out, const void* positions, int64_t pos_stride,
                        const uint64_t* turns, const int32_t* axis, int64_t n_tokens,
                        int64_t n_q_heads, int64_t n_k_heads, int64_t head_dim, int64_t rot_dim,
                        int64_t n_axes, int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                        int64_t k_out_stride, float eps, float weight_offset, uint32_t flags,
                        cudaStream_t stream);

/*
 * A paged cache of keys and values in E4M3 codes, with one fp32 scale for
 * every block of RMSATTN_BLOCK tokens and head: value = code * scale.
 *
 *   k, v             [n_pages, n_kv_heads, page_size, head_dim] bytes, pages
 *                    page_stride bytes apart, 16-byte aligned
 *   k_scale, v_scale [n_pages, n_kv_heads, page_size / RMSATTN_BLOCK] fp32,
 *                    pages scale_stride floats apart (n_pages * scale_stride
 *                    < 2^32, else RMSN_EUNSUPPORTED)
 *
 * Scales are finite and not negative (the append makes no others).
 * head_dim is 64, 128 or 256; page_size a multiple of RMSATTN_BLOCK up to
 * 65536.  A block table row lists a sequence's pages in order: token i is
 * row i % page_size of page block_table[seq][i / page_size].
 */
#define RMSATTN_BLOCK 16

typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t n_pages;
    int64_t page_stride;  /* bytes, a multiple of 16 */
    int64_t scale_stride; /* floats */
    int32_t n_kv_heads;
    int32_t page_size;
    int32_t head_dim;
    int32_t reserved; /* 0 */
} rmsattn_cache;

/*
 * Append new keys and values.  Sequence s holds lengths[s] tokens and gets
 * the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 of k and v behind them
 * (cu_seqlens NULL: row s alone, n_tokens == n_seqs).  Per block of 16 tokens
 * and head that gets a token, for k and v alike:
 *
 *   a  = max over the block's new elements of min(|x|, FLT_MAX), NaN left out
 *   s' = max(s, a / 448), s the block's scale before, 0 if none of its tokens
 *        is older; at least 2^-126 unless a and s are 0
 *   new codes  E4M3_RN_SATFINITE(x * r) with r = RN(1 / s') (r = 0 if s' = 0)
 *   old codes, where s' > s: E4M3_RN_SATFINITE(code * RN(s * r))
 *
 * An infinity saturates to the largest code, a NaN keeps its NaN code.  Every
 * other byte of the cache stays as it is.  lengths is not changed.  A
 * sequence with lengths[s] < 0 is left out (a padded batch's row).  A token
 * past the table's width, or in a page outside [0, n_pages), is dropped and
 * sets bit 2 (value 4) of the status word; a sequence whose rows lie outside
 * [0, n_tokens) is left out.  In one call no page may get tokens by two table
 * entries, of two sequences or of one.
 *
 *   k, v        [n_tokens, n_kv_heads, head_dim] bf16 / fp16 / fp32, token
 *               strides in elements (heads back to back)
 *   block_table [n_seqs, table_width] int32, rows table_stride apart
 *   lengths     [n_seqs] int32; cu_seqlens [n_seqs + 1] int32, non-decreasing
 */
int rmsattn_kv_append(const rmsattn_cache* cache, const void* k, const void* v, int64_t k_stride,
                      int64_t v_stride, const int32_t* block_table, int64_t table_stride,
                      int64_t table_width, const int32_t* lengths, const int32_t* cu_seqlens,
                      int64_t n_tokens, int64_t n_seqs, uint32_t flags, cudaStream_t stream);

/*
 * Attention of n_queries tokens per sequence over the cache (1 for a decode
 * step, a few for drafted tokens; at most RMSATTN_MAX_QUERIES).  lengths[s]
 * counts the cached tokens, the queries' own among them: query i of sequence
 * s sits at position lengths[s] - n_queries + i and sees token j when
 *
 *   j <= position  and  (window == 0 or j > position - window or j < sinks)
 *
 *   out = sum_j softmax_j(scale * q . k_j) v_j     (0 where nothing is seen)
 *
 * Query head h reads key head h / (n_q_heads / n_kv_heads).  A row of q is held
 * in fp16 times a power of two: each element exactly, or to within 2^-32 of the
 * row's largest.  Its products with the codes are exact in fp32 sums; scores
 * (finite below 3.4e38), softmax statistics and the output sum are fp32; the
 * weights are rounded to fp16 (2^-11 of their value, or 2^-33 of the row's
 * largest) for the second product, whose value scales are applied in fp32 (one
 * below 2^-118 keeps 16 bits).  An infinity or NaN in a row of q gives NaN
 * wherever that row sees a token.  Tokens past lengths[s], and tokens that no
 * query of the sequence sees, have no influence, whatever their codes are; one
 * that another query of the sequence sees may change a result's last roundings.
 * A page outside [0, n_pages), or past the table's width, is left out and sets
 * bit 2 (value 4) of the status word.
 *
 *   q, out      [n_seqs, n_queries, n_q_heads, head_dim] bf16 / fp16, tokens
 *               q_stride / out_stride elements apart, heads back to back, 16-byte
 *               aligned with strides of whole 16-byte vectors
 *   workspace   rmsattn_kv_attention_workspace(...) bytes on the device, 16-byte
 *               aligned, used by this call alone until it has finished (may be
 *               NULL where that is 0)
 */
#define RMSATTN_MAX_QUERIES 32

int rmsattn_kv_attention(const void* q, const rmsattn_cache* cache, const int32_t* block_table,
                         int64_t table_stride, int64_t table_width, const int32_t* lengths,
                         void* out, int64_t q_stride, int64_t out_stride, int64_t n_seqs,
                         int64_t n_queries, int64_t n_q_heads, float scale, int64_t window,
                         int64_t sinks, void* workspace, int64_t workspace_bytes, uint32_t flags,
                         cudaStream_t stream);

/* Bytes of workspace that rmsattn_kv_attention needs for these sizes on the
 * current device (>= 0), or a negative rmsn_status.  max_tokens: what a table
 * row holds, table_width * page_size. */
int64_t rmsattn_kv_attention_workspace(int64_t n_seqs, int64_t n_queries, int64_t n_q_heads,
                                       int64_t n_kv_heads, int64_t head_dim, int64_t max_tokens,
                                       int64_t window, int64_t sinks);

/* Status word of this library's kernels on the current device: bit 2 (value
 * 4) is set when a block table named a page outside the cache or a token lay
 * past the table.  Reads synchronously, behind the legacy default stream's work:
 * synchronise with streams made non-blocking (PyTorch's own) first.  `clear` !=
 * 0 resets the word. */
int rmsattn_read_status(uint32_t* status, int clear);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_ATTN_GB300_H */
