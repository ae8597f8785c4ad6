/*
 * tree_kv4.h — C ABI of a KV cache held in 4 bits and the verify step on it,
 * on NVIDIA GB300 (sm_103a): writing rows, committing an accepted path,
 * reading rows back, and the tree-verify attention.
 *
 * Format.  A cached value is (u - 8) * s with a 4-bit u in 0..15 and a scale
 * s = 2^(e - 15) * (1 + m / 8) held in one byte e * 8 + m (e 0..31, m 0..7).
 * K has one scale per position and 32 channels, V one per position and KV
 * head.  With 3-bit magnitudes and 4-bit scale significands every value is
 * exact in bf16.  Writing takes the smallest scale with 7 s >= the largest
 * magnitude of its group (the largest scale if none), and
 * u = 8 + clamp(round(x / s), -7, 7), ties to even: the error is at most
 * s / 2 for magnitudes up to 7 * 122880.  NaN is written as 0; an infinity
 * takes the largest scale and 7 steps.
 *
 * Layout.  16 consecutive positions of one KV head are one block:
 *   K block, 8.5 d bytes: for each 32 channels c, 16 positions x 16 bytes;
 *                         then for each 32 channels 16 scale bytes (by position)
 *   V block, 8 d + 16 bytes: for each channel 8 bytes holding its 16
 *                         positions; then 16 scale bytes (by position)
 * Eight values are one little-endian 32-bit word: value 2 j at bits 4 j ..
 * 4 j + 3, value 2 j + 1 at bits 16 + 4 j .. 19 + 4 j (8 channels of K, 8
 * positions of V).  The blocks are
 *   contiguous: [B, Hkv, capacity / 16, block bytes]
 *   paged:      [num_pages, Hkv, block bytes], page_table as in tree_verify.h
 * so a K value takes 4.25 bits and a V value 4 + 8 / d.
 * The capacity is a multiple of 16 in both cases.
 *
 * Rounding.  Cached values are exact in both types.  fp32 calls are computed in
 * fp32.  bf16 calls accumulate, and take the softmax and the partial results,
 * in fp32; each softmax weight, times its position's V scale, is rounded to
 * bf16 (2^-8 of it at most) before it multiplies the steps u - 8 of V,
 * while the sum that divides keeps the unrounded weights.  These weights are
 * relative to one of the row's scores, not always its largest, and reach 2^60:
 * V of the tree should stay below 2^60 in magnitude there.
 *
 * desc->dtype is the type of queries, of the tree's K/V and of the rows
 * written and read.  The calls on the cache alone (tv_kv4_cache_bytes,
 * tv_kv4_append, tv_kv4_read) have no tree: the descriptor's max_nodes and
 * total_rows are not looked at.  Everything else follows tree_verify.h: buffers are the
 * caller's, device pointers 16-byte aligned, host errors before anything is
 * enqueued, device faults OR-ed into *d_status.
 */
#ifndef TREE_KV4_H
#define TREE_KV4_H

#include "tree_verify.h"
#include "tree_window.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the K and of the V cache of a descriptor (contiguous: batch and
 * capacity; paged: num_pages).  TV_ERR_SHAPE when the capacity is not a
 * multiple of 16. */
int tv_kv4_cache_bytes(const tv_desc* desc, int64_t* k_bytes, int64_t* v_bytes);

/* Writes rows into the cache.  Sequence b's rows are
 * [d_row_offsets[b], d_row_offsets[b + 1]) of d_k and d_v [Hkv, rows, d]
 * (dtype); row i of the sequence goes to position d_start[b] + i.  Other
 * positions keep their bytes.  max_rows: host upper bound on a sequence's
 * rows (sizes the grid).  A sequence whose offsets are invalid
 * (TV_DEV_BAD_OFFSETS), whose start is negative (TV_DEV_BAD_PREFIX) or whose
 * rows do not fit (TV_DEV_CAPACITY) is skipped; rows on an invalid page are
 * skipped (TV_DEV_BAD_PAGE).  A sequence may have no rows (equal offsets): it
 * reads and writes nothing, and its page-table entries may hold anything.  No
 * two sequences may write the same block.
 * Errors: TV_ERR_SHAPE (rows < 0, max_rows < 0, or too many blocks),
 * TV_ERR_NULL, TV_ERR_ALIGN, TV_ERR_PAGED, TV_ERR_OVERFLOW, TV_ERR_CUDA.
 * rows = 0 or max_rows = 0 enqueues nothing (d_k and d_v may then be NULL). */
int tv_kv4_append(const tv_desc* desc, int64_t rows, int64_t max_rows, const void* d_k, const void* d_v,
                  const int32_t* d_row_offsets, const int32_t* d_start, void* d_k4, void* d_v4,
                  const int32_t* d_page_table, int32_t* d_status, void* stream);

/* The reverse of tv_kv4_append: the values the cache stands for at positions
 * d_start[b] + i into rows of d_k and d_v [Hkv, rows, d] (dtype; exact in
 * both).  Rows of skipped sequences and pages keep their contents. */
int tv_kv4_read(const tv_desc* desc, int64_t rows, int64_t max_rows, const void* d_k4, const void* d_v4,
                const int32_t* d_page_table, const int32_t* d_row_offsets, const int32_t* d_start, void* d_k,
                void* d_v, int32_t* d_status, void* stream);

/* tree_accept_commit_argmax (tree_verify.h) with a 4-bit cache: the walk on
 * the given target argmax, then the accepted rows of the tree's K/V are
 * written at positions P_b .. P_b + k, and prefix_len advances.  Same
 * outputs, skips and errors as there. */
int tree_accept_commit_argmax_kv4(const tv_desc* desc, const int32_t* d_argmax, const int32_t* d_draft_tokens,
                                  const int32_t* d_parents, const int32_t* d_node_offsets, const void* d_k_tree,
                                  const void* d_v_tree, void* d_k4, void* d_v4, const int32_t* d_page_table,
                                  int32_t* d_prefix_len, int32_t* d_accept_len, int32_t* d_path, int32_t* d_tokens,
                                  int32_t* d_status, void* stream);

/* Scratch bytes and plan of tree_verify_attn_kv4 (win may be NULL).  Plan
 * kernel 0: CUDA cores (fp32, or more than 64 query heads per KV head);
 * 4: tcgen05 with the cache expanded into tensor memory; 5: up to 8 rows per
 * KV head (max_nodes * Hq / Hkv), the cache expanded in registers. */
int tv_kv4_workspace_size(const tv_desc* desc, const tv_window* win, size_t* bytes);
int tv_kv4_attn_plan(const tv_desc* desc, const tv_window* win, tv_plan* plan);

/* tree_verify_attn with the prefix in a 4-bit cache and the tree's own K/V
 * in dtype.  win NULL: the whole prefix is visible (d_depth may then be
 * NULL); otherwise as in tree_verify_attn_window. */
int tree_verify_attn_kv4(const tv_desc* desc, const tv_window* win, const void* d_q, const void* d_k4,
                         const void* d_v4, const int32_t* d_page_table, const int32_t* d_prefix_len,
                         const int32_t* d_node_offsets, const void* d_k_tree, const void* d_v_tree,
                         const uint64_t* d_anc, const int32_t* d_depth, void* d_out, void* d_workspace,
                         size_t workspace_bytes, int32_t* d_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TREE_KV4_H */
