/*
 * tree_window.h — C ABI of tree-verify attention over a sliding window with
 * attention sinks, on NVIDIA GB300 (sm_103a).
 *
 * What it computes: tree_verify_attn (tree_verify.h) where a row no longer
 * sees its whole past.  Tree row r of sequence b, at position
 * p = prefix_len[b] + depth[r], sees a key at position t iff
 *     t < sinks   or   p - t < window,
 * among the keys tree_verify_attn shows it: the prefix positions
 * 0 .. prefix_len[b] - 1, and its ancestors and itself (tree node a is at
 * position prefix_len[b] + depth[a]).  window >= 1, so a row always sees
 * itself; window >= prefix_len + 64 is the whole past.  Positions outside
 * every row's view are not read, so the call costs what the sinks and the
 * window hold, whatever the prefix length.
 *
 * Conventions are those of tree_verify.h.  The cache keeps its positions:
 * a key that left the window keeps its place and is not read again unless it
 * is a sink, so a paged cache may free its page.  The page table's entries of
 * 16-position pages that no row sees (wholly in [sinks, prefix_len - window
 * + 1)) are not read and may hold anything, and so may every cache row that no
 * row sees.  V that some rows of a sequence see must be finite for the others.
 *
 * Rounding.  fp32 calls are computed in fp32.  bf16 calls accumulate, and take
 * the softmax and the partial results, in fp32; each softmax weight is rounded
 * to bf16 (2^-8 of it at most) before it multiplies V, while the sum
 * that divides keeps the unrounded ones.
 */
#ifndef TREE_WINDOW_H
#define TREE_WINDOW_H

#include "tree_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tv_window {
  int64_t window;   /* positions a row sees up to and including its own, >= 1 */
  int64_t sinks;    /* first positions that every row sees, >= 0 */
} tv_window;

/* Bytes of scratch tree_verify_attn_window needs (256-byte aligned; any
 * contents), and the plan it runs (kernel 0 or 1 of tv_plan).  Errors: those
 * of tv_workspace_size, TV_ERR_NULL, TV_ERR_SHAPE (window < 1, sinks < 0). */
int tv_window_workspace_size(const tv_desc* desc, const tv_window* win, size_t* bytes);
int tv_window_attn_plan(const tv_desc* desc, const tv_window* win, tv_plan* plan);

/* tree_verify_attn over the window: every argument as there, and
 *   win, the window and sinks of every row, and
 *   d_depth [total_rows] int32, from tv_build_tree_mask.
 * Types, layouts, caches and errors are those of tree_verify_attn. */
int tree_verify_attn_window(const tv_desc* desc, const tv_window* win, const void* d_q, const void* d_k_cache,
                            const void* d_v_cache, const int32_t* d_page_table, const int32_t* d_prefix_len,
                            const int32_t* d_node_offsets, const void* d_k_tree, const void* d_v_tree,
                            const uint64_t* d_anc, const int32_t* d_depth, void* d_out, void* d_workspace,
                            size_t workspace_bytes, int32_t* d_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TREE_WINDOW_H */
