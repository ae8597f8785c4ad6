/*
 * tree_prompt.h — C ABI of the prompt's way into the cache, on NVIDIA GB300
 * (sm_103a): what a serving loop runs before the first verify step, and
 * whenever a sequence gets a new turn.
 *
 *   tv_prompt_rope_store  rotates the rows' queries and keys at their
 *                         positions, and writes keys and values head-major
 *                         into rows and to their positions of the cache
 *   tv_prompt_attn        causal attention of those rows: row i of sequence b
 *                         stands at position P_b + i and sees the committed
 *                         prefix (positions 0 .. P_b - 1 of the cache) and
 *                         rows 0 .. i of its own sequence
 *
 * Rows.  Sequence b's rows are [d_row_offsets[b], d_row_offsets[b + 1]) of
 * `rows` packed rows, n_b of them, 0 <= n_b <= max_rows (a host upper bound
 * that sizes the grid and the scratch).  A sequence may have no rows: nothing
 * of it is read or written.  Rows at or past d_row_offsets[batch] belong to no
 * sequence (a padded batch): the outputs' rows there are left as they were.
 * P_b = d_prefix_len[b], at most max_prefix; n_b has no bound of its own, so a
 * prompt may come whole or in chunks, and a chunk of up to 64 rows is what a
 * chain of tree rows is to tree_verify_attn.
 *
 * Layouts, types, pages, heads and scale are those of tree_verify.h:
 *   q, out         [rows, Hq, d]
 *   k/v rows       [Hkv, rows, d]
 *   k/v cache      contiguous [B, Hkv, capacity, d] or paged [num_pages, Hkv, 16, d]
 * The descriptor's max_nodes and total_rows are not looked at (there is no
 * tree).  The attention never reads cache positions >= P_b, so the two calls
 * may come in either order once the rows are written, and prefix_len advances
 * when every layer is done (tv_prompt_rope_store gives the new lengths).  Where
 * no sequence has a prefix (max_prefix = 0) the attention takes NULL for the
 * cache and the page table: a prompt into a cache of another form, such as the
 * 4-bit cache of tree_kv4.h, whose tv_kv4_append takes the same rows.
 *
 * Conventions are those of tree_verify.h: the caller's buffers, 16-byte
 * aligned device pointers, host errors before anything is enqueued, device
 * faults OR-ed into *d_status, nothing allocated or synchronised,
 * deterministic results.  rows = 0 or max_rows = 0 enqueues nothing: the
 * pointers are then not looked at, and no output is written, the new lengths
 * neither.
 *
 * Device faults of both calls: where a sequence's offsets are invalid
 * (TV_DEV_BAD_OFFSETS) it is skipped, and what the call leaves in the outputs of
 * the others is undefined; a prefix length out of range is clamped
 * (TV_DEV_BAD_PREFIX).
 */
#ifndef TREE_PROMPT_H
#define TREE_PROMPT_H

#include "tree_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rotation (tree_rope.h's: NeoX pairs over the whole head, angle
 * p * theta^(-2j/d) at position p = P_b + i) of every query and key head, and
 * the writes:
 *   d_q_out [rows, Hq, d] (may equal d_q_in);
 *   d_k_rows, d_v_rows [Hkv, rows, d], both or neither (NULL);
 *   d_k_cache, d_v_cache, position P_b + i, both or neither (NULL), with
 *   d_page_table when the cache is paged;
 *   d_new_prefix_len [B] or NULL: P_b + n_b, or d_prefix_len[b] as it was
 *   where the sequence is skipped, or where the sum passes 2^31 - 1
 *   (TV_DEV_CAPACITY).  It must not be d_prefix_len (TV_ERR_SHAPE).
 * d_q_in [rows, Hq, d], d_k_in and d_v_in [rows, Hkv, d].  No other buffers may
 * overlap.  With a cache, a sequence whose rows do not fit (P_b + n_b >
 * capacity: TV_DEV_CAPACITY) is skipped whole, and so is one whose prefix
 * length is out of range (TV_DEV_BAD_PREFIX; without a cache it is clamped);
 * cache rows on an invalid page are not written (TV_DEV_BAD_PAGE), the other
 * outputs are.  No two sequences may write one page.
 * Precision: each angle is reduced in 64 bits, its sine and cosine taken in
 * fp32, the rotation in fp32, then rounded once to the type; values are copied.
 * Errors: TV_ERR_NULL, TV_ERR_SHAPE (rows or max_rows negative or rows >= 2^31,
 * theta not finite or <= 1), TV_ERR_ALIGN, TV_ERR_PAGED, TV_ERR_OVERFLOW, the
 * descriptor's, TV_ERR_CUDA. */
int tv_prompt_rope_store(const tv_desc* desc, int64_t rows, int64_t max_rows, double theta, const void* d_q_in,
                         const void* d_k_in, const void* d_v_in, const int32_t* d_prefix_len,
                         const int32_t* d_row_offsets, void* d_q_out, void* d_k_rows, void* d_v_rows,
                         void* d_k_cache, void* d_v_cache, const int32_t* d_page_table, int32_t* d_new_prefix_len,
                         int32_t* d_status, void* stream);

/* Bytes of scratch tv_prompt_attn needs (256-byte aligned; any contents; one
 * call at a time).  Few rows over many keys are split over the keys and many
 * rows are not, so a smaller call may need more than a larger one: the size is
 * that of these rows, max_rows and max_prefix alone.  And the plan it runs: kernel 6 tcgen05 with two query tiles a
 * CTA (bf16, head_dim 128), 7 tcgen05 on CTA pairs (bf16, 256 and 512), 8
 * tcgen05 on numbers in three bf16 parts (fp32; bf16 with more than 128 query
 * heads a KV head or a cache of 2^31 rows); chunk and num_splits count keys in
 * tiles of 128 (prefix and rows each rounded up).  Kernel 8 keeps 12 bytes a
 * value of K and V of max_prefix and the rows in the scratch. */
int tv_prompt_workspace_size(const tv_desc* desc, int64_t rows, int64_t max_rows, size_t* bytes);
int tv_prompt_attn_plan(const tv_desc* desc, int64_t rows, int64_t max_rows, tv_plan* plan);

/* out[r, h, :] = sum_j softmax_j(scale * q[r,h,:] . k_j) v_j over the keys row
 * r sees.  fp32 inputs are computed to fp32 accuracy: each
 * number as the sum of three bf16 ones (exact below 2^127 in magnitude; seen K
 * and V must be finite), six products of them on the tensor cores, sums in fp32,
 * the sum over the keys rounded to nearest from tile to tile.  bf16 inputs are
 * multiplied in bf16 with fp32 accumulation, an fp32 softmax and fp32
 * partials; each weight is rounded to bf16 (2^-8 of it at most) before it
 * multiplies V, while the sum that divides keeps the unrounded ones.
 * d_k_cache and d_v_cache may be NULL when max_prefix = 0.  The cache, q and
 * the rows are only read.  A row's answer does not depend on other sequences'
 * rows or on cache positions past its prefix; V of a later row of its own
 * sequence must be finite (a weight of 0 multiplies it).  bf16: a score of -inf
 * weighs nothing, and a row all of whose scores are -inf gives zeros.  A page id
 * out of range reads as zeros (TV_DEV_BAD_PAGE). */
int tv_prompt_attn(const tv_desc* desc, int64_t rows, int64_t max_rows, const void* d_q, const void* d_k_cache,
                   const void* d_v_cache, const int32_t* d_page_table, const int32_t* d_prefix_len,
                   const int32_t* d_row_offsets, const void* d_k_rows, const void* d_v_rows, void* d_out,
                   void* d_workspace, size_t workspace_bytes, int32_t* d_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TREE_PROMPT_H */
