/*
 * rmsnorm_attn.h -- C ABI of the GB300 (sm_103a) attention-path operators
 * that stand next to the QK norm of rmsnorm.h: rotary positions with several
 * axes fused with that norm, the append of keys and values to a paged 8-bit
 * cache, the attention that reads it (with a form for sequences that share a
 * long prefix), the page plan of a serving step, and the norms at a block's end.
 * Built into a library of its own
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

/*
 * The same attention where groups of sequences share a long first part (a system
 * prompt, a document): the shared tokens are read once for a group, and all of
 * its queries are multiplied with them on the tensor cores.  The result is that
 * of rmsattn_kv_attention without window and sinks, up to the order of sums.  Its
 * four or five launches take some 25 us whatever the sizes: it is the faster one where
 * the rows of all sequences, prefixes counted for each, are more than about 200 MB
 * at head_dim 64 and 128, or 300 MB at 256 (2 n_kv_heads (head_dim + 1/4) bytes a token).
 *
 *   group_cu       [n_groups + 1] int32, non-decreasing: group g is the sequences
 *                  group_cu[g] .. group_cu[g + 1] - 1; sequences of no group
 *                  share nothing.  NULL: one group of all (n_groups 1, or 0)
 *   prefix_lengths [n_groups] int32: the first tokens that are the same for all
 *                  of the group, in the same pages (the rows of the block table
 *                  begin with the same entries).  Any length, 0 among them; whole
 *                  blocks of RMSATTN_BLOCK tokens are shared, the rest is read by
 *                  each sequence.
 *
 * block_table and lengths count the shared tokens too, as everywhere.  A sequence
 * whose first query does not see all of the prefix, one of length 0 among them,
 * and one that is alone in its group shares nothing: it reads its own row.  The
 * shared pages are those of the group's first sequence that shares.  Borders that
 * decrease or leave [0, n_seqs] share nothing, and set bit 2 (value 4) of the
 * status word.
 *
 * The second product's weights are rounded to fp16 after they have been
 * multiplied with the significand of their block's value scale (2^-11 of their
 * value, or 2^-34 of the row's largest); the scale's power of two goes to the
 * codes, which stay exact.
 *
 *   workspace   rmsattn_kv_prefix_attention_workspace(...) bytes on the device,
 *               32-byte aligned, used by this call alone until it has finished
 */
int rmsattn_kv_prefix_attention(const void* q, const rmsattn_cache* cache, const int32_t* block_table,
                                int64_t table_stride, int64_t table_width, const int32_t* lengths,
                                const int32_t* prefix_lengths, const int32_t* group_cu, int64_t n_groups,
                                void* out, int64_t q_stride, int64_t out_stride, int64_t n_seqs,
                                int64_t n_queries, int64_t n_q_heads, float scale, void* workspace,
                                int64_t workspace_bytes, uint32_t flags, cudaStream_t stream);

/* Bytes of workspace for these sizes on the current device (>= 0), or a negative
 * rmsn_status.  max_tokens: table_width * page_size.  It grows with the rows
 * n_seqs * n_queries * n_q_heads, by about 8 * head_dim + 16 bytes each, and with the
 * groups by up to 28 * n_kv_heads * (head_dim + 2) bytes each, over some 5 to 25 MB. */
int64_t rmsattn_kv_prefix_attention_workspace(int64_t n_seqs, int64_t n_queries, int64_t n_q_heads,
                                              int64_t n_kv_heads, int64_t head_dim, int64_t max_tokens,
                                              int64_t n_groups);

/*
 * A serving step's plan from the requests' lengths.  Sequence s holds lengths[s]
 * tokens and gets new_tokens[s] more, the next new_tokens[s] rows of the step's
 * batch of n_rows (as rmsattn_kv_append takes them); a negative new_tokens[s]
 * says that it is finished, a negative lengths[s] that there is no sequence s.
 *
 *   own(s)  = ceil(lengths[s] / page_size) pages, need(s) with the new tokens
 *   returned, in the sequences' order: the pages [shared_pages[s], own(s)) of the
 *     rows of finished sequences (within the table's width); they go behind the
 *     n_free first entries of free_pages: F = n_free + returned, at most n_pages
 *   taken, in the sequences' order: need(s) - own(s) pages; the k-th of all that
 *     is taken is entry F - 1 - k, and becomes block_table[s][own(s) ...]
 *   left out: a sequence whose pages outrun F (with all pages asked for before
 *     it) or the table's width, whose rows outrun n_rows, or whose tokens outrun
 *     31 bits.  It takes nothing, and its table row stays as it is.
 *
 * Results, all int32 but slots:
 *   cu_seqlens [n_seqs + 1]  the sequences' first rows, and the end (at most n_rows)
 *   positions  [n_rows]      lengths[s] + i for a sequence's row i; 0 behind the last
 *   slots      [n_rows]      int64: page * page_size + row in the page; -1 behind
 *                            the last row and for a sequence that is left out
 *   rows       [n_rows]      the row's sequence; -1 behind the last
 *   before     [n_seqs]      lengths[s], what rmsattn_kv_append takes; -1 for a
 *                            sequence that is left out, finished or not there
 *   after      [n_seqs]      tokens behind the step, what the attention takes: 0
 *                            for a finished sequence, lengths[s] for one left out
 *   n_free_out [1]           free pages behind the step, F - taken
 * and in place block_table (the new entries alone) and free_pages (the returned
 * pages among its first n_free_out entries).  lengths and n_free are not changed,
 * so the same call gives the same results again; a program goes on with `after` and
 * n_free_out.  What is written (results, workspace, free_pages, block_table) shares no
 * byte with each other or with lengths, new_tokens, shared_pages and n_free: such a
 * call is refused.
 *
 * free_pages holds n_pages entries, of which the first n_free (kept within
 * [0, n_pages]) count; page numbers outside [0, n_pages) and more returned pages
 * than free_pages holds set bit 2 (value 4) of the status word (slots are then -1).
 * shared_pages may be NULL (0); page_size as in rmsattn_cache.  positions, rows
 * and slots are 16-byte aligned.
 */
int rmsattn_pages_step(int32_t* free_pages, int64_t n_pages, const int32_t* n_free,
                       int32_t* block_table, int64_t table_stride, int64_t table_width,
                       const int32_t* lengths, const int32_t* new_tokens, const int32_t* shared_pages,
                       int64_t n_seqs, int64_t page_size, int64_t n_rows, int32_t* cu_seqlens,
                       int32_t* positions, int64_t* slots, int32_t* rows, int32_t* before,
                       int32_t* after, int32_t* n_free_out, void* workspace, int64_t workspace_bytes,
                       uint32_t flags, cudaStream_t stream);

/* Bytes of workspace that rmsattn_pages_step needs (16-byte aligned; 0 up to 2048
 * sequences), or a negative rmsn_status. */
int64_t rmsattn_pages_workspace(int64_t n_seqs);

/*
 * The end of a block and the begin of the next, for each row of `hidden` elements:
 *
 *   p = (post_weight + weight_offset) * (x * rsqrt(mean(x^2) + eps))
 *   h = RN(residual_scale * residual + gate * p)     -> residual_out
 *   y = (weight + weight_offset) * (h * rsqrt(mean(h^2) + eps))   -> out
 *
 * in fp32, h rounded once to the residual's type, y (of the rounded h) once to
 * x's; with RMSATTN_OUT_FP8, out holds E4M3_RN_SATFINITE(y * (448 / max|y|)) and
 * out_scale max|y| / 448 (a row of zeros: codes and scale 0; where 448 / max|y| lies
 * outside fp32's range, both factors are taken times a power of two first).
 *
 *   x            [n_tokens, hidden] bf16 / fp16 / fp32, weights [hidden] of its type
 *                or NULL (1, without the offset)
 *   residual     [n_tokens, hidden] of x's type, or fp32 with RMSN_RESIDUAL_F32
 *                (bf16 / fp16 x); residual_out the same
 *   out          of x's type, or bytes
 *   gate         NULL (1); or rows of x's type gate_stride elements apart:
 *                gate_stride 0, n_gates 1: one row for all; n_gates == n_tokens: a
 *                row each; with gate_index [n_tokens], token t takes row
 *                gate_index[t] of n_gates, and one with a negative index (a row
 *                behind the last sequence) is left out, out, residual_out and
 *                out_scale untouched, or zeros there with RMSATTN_ZERO_OUT,
 *                RMSATTN_ZERO_RESIDUAL and RMSATTN_ZERO_SCALE (outputs that nothing
 *                was written to before).  An index >= n_gates is left out too, and sets
 *                bit 2 (value 4) of the status word.  Where n_tokens or n_gates is 0, the
 *                pointers of what is empty may be NULL.
 *
 * An output may be x, residual, or a gate row for each token (gate_stride ==
 * hidden), where that has the output's type; any other memory that an output shares
 * with an input or with another output is refused.
 *
 * Sums of squares are fp32: rows need sum(x^2), sum(h^2) < FLT_MAX.  Rows, gates
 * and weights are contiguous.  Vectors of eight elements are used where x, residual,
 * out and residual_out each begin on such a vector, for any hidden up to 16384 (16377
 * where rows, gates or weights begin off the vectors); other calls go element by
 * element, and take about four times as long.
 */
#define RMSATTN_OUT_FP8 0x8000u
#define RMSATTN_ZERO_OUT 0x10000u
#define RMSATTN_ZERO_RESIDUAL 0x20000u
#define RMSATTN_ZERO_SCALE 0x40000u

int rmsattn_block_norms(const void* x, const void* residual, const void* post_weight,
                        const void* weight, const void* gate, int64_t gate_stride,
                        const int32_t* gate_index, int64_t n_gates, void* out, void* residual_out,
                        float* out_scale, int64_t n_tokens, int64_t hidden, float eps,
                        float residual_scale, float weight_offset, uint32_t flags,
                        cudaStream_t stream);

/* Status word of this library's kernels on the current device: bit 2 (value
 * 4) is set when a block table named a page outside the cache or a token lay
 * past the table (and by what the plan and the norms say above); bit 0 (value 1)
 * when a wait inside rmsattn_kv_prefix_attention ran out after about a second
 * (its result is then not to be used; a defect, no input leads there).  Reads
 * synchronously, behind the legacy default stream's work: synchronise with
 * streams made non-blocking (PyTorch's own) first.  `clear` != 0 resets the word. */
int rmsattn_read_status(uint32_t* status, int clear);

/* Testing hook for the bounded waits inside rmsattn_kv_prefix_attention (not needed in
 * normal use).  Sets, for calls that follow on the current device, after how many SM
 * clock cycles a wait gives up: its block then stops, waits for what it has in flight
 * (with the default bound), and bit 0 of the status word is set; the call's result is not
 * to be used.  0 restores the default (about one second); a negative value makes a wait
 * give up as soon as its barrier has been tried, so that the give-up path runs on a
 * healthy GPU. */
int rmsattn_set_wait_limit(int64_t cycles);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_ATTN_GB300_H */
