/*
 * tree_logits.h — C ABI of the control of the target's logits at every tree
 * row, on NVIDIA GB300 (sm_103a): penalties for repeated tokens, a bias for
 * chosen tokens and a grammar's mask, between the lm_head and
 * tree_accept_commit / tree_accept_commit_sampled (tree_verify.h).
 *
 * What it computes.  For tree row r of sequence b and token v, with x the
 * logit, n = emitted(b, v) + the drafts equal to v on the path from the root
 * to row r (its own draft included, the root's not: the root is the last
 * emitted token and counted already), and seen = prompt(b, v) or n > 0:
 *     if seen:   x = x > 0 ? x / rho_b : x * rho_b       (repetition)
 *     x = x - phi_b * n - pi_b * [n > 0]                 (frequency, presence)
 *     x = x + bias_b(v)
 *     if the mask forbids v at row r:  x = -inf
 * in fp32, in this order, rounded once to the logits' type.  So every tree row
 * is steered as plain decoding would steer it after that row's path.  A row
 * whose mask allows nothing is -inf everywhere (its argmax is token 0).  NaN
 * stays NaN where it is allowed, and -inf stays -inf.
 *
 * Counts.  One 16-bit word per sequence and token, in rows of
 * (vocab + 7) / 8 * 8 words: bit 15 is set when the token stands in the
 * prompt, bits 0 - 14 hold how often it was emitted (no more than 32767 are
 * counted).  All zeros is a new sequence.  tv_token_counts_add counts a
 * prompt's tokens, the token that the prompt's last row gave (the first tree's
 * root) and each step's emitted ones.
 *
 * Conventions are those of tree_verify.h.
 */
#ifndef TREE_LOGITS_H
#define TREE_LOGITS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* device status bit (the others are TV_DEV_* of tree_verify.h and tree_expand.h) */
enum {
  TV_DEV_BAD_TOKEN = 256   /* a token outside [0, vocab): it is left out */
};

typedef struct tv_logits_desc {
  int32_t batch;          /* B >= 1 sequences */
  int32_t vocab;          /* V, 1..2^30 */
  int32_t max_nodes;      /* upper bound on a sequence's tree rows, 1..64 */
  int32_t total_rows;     /* tree rows, batch..batch * max_nodes */
  int32_t logits_dtype;   /* TV_F32 or TV_BF16 (tree_verify.h) */
  int32_t biases;         /* entries of the bias lists over all sequences, >= 0; ignored without them */
} tv_logits_desc;

/* Adds tokens to the counts: as prompt tokens (prompt != 0) or as emitted ones.
 * d_offsets [B+1] int32: sequence b's tokens are [d_offsets[b],
 * d_offsets[b+1]) of d_tokens, `tokens` of them in all; or NULL: they are
 * d_tokens[b * tokens .. b * tokens + tokens - 1], as the [B, max_nodes] rows
 * that tree_accept_commit leaves.  Negative tokens are padding and skipped;
 * tokens >= vocab are skipped with TV_DEV_BAD_TOKEN.  Invalid offsets skip
 * their sequence (TV_DEV_BAD_OFFSETS).  tokens = 0 enqueues nothing.
 * Only batch and vocab of the descriptor are looked at.
 * Errors: TV_ERR_NULL, TV_ERR_SHAPE, TV_ERR_OVERFLOW, TV_ERR_ALIGN, TV_ERR_CUDA. */
int tv_token_counts_add(const tv_logits_desc* desc, const int32_t* d_tokens, const int32_t* d_offsets,
                        int64_t tokens, int32_t prompt, uint16_t* d_counts, int32_t* d_status, void* stream);

/* The logits of every tree row, from d_logits [total_rows, vocab] to d_out
 * (the same type; d_out may equal d_logits, else they must not overlap).
 *   d_counts, d_penalties [B, 3] float (rho_b > 0, phi_b, pi_b): both, or NULL
 *     both (no penalties);
 *   d_bias_offsets [B+1] int32, d_bias_tokens, d_bias_values (int32, float):
 *     sequence b's biases are [d_bias_offsets[b], d_bias_offsets[b+1]); the
 *     three, or NULL all.  A token listed twice takes the later value; tokens
 *     outside [0, vocab) are left out (TV_DEV_BAD_TOKEN); offsets that decrease
 *     or leave [0, biases] leave the sequence's biases out (TV_DEV_BAD_OFFSETS);
 *   d_mask [total_rows, (vocab + 31) / 32] uint32 or NULL: token 32 w + i is
 *     allowed iff bit i of word w is set;
 *   d_draft_tokens [total_rows], d_anc [total_rows] uint64 (from
 *     tv_build_tree_mask): the rows' paths; both, or NULL both (no drafts are
 *     counted).  They matter only with d_counts.  Draft tokens outside
 *     [0, vocab) are not counted.
 * A sequence whose node offsets are invalid is skipped (TV_DEV_BAD_OFFSETS):
 * its rows of d_out keep their contents.
 * Errors: TV_ERR_NULL, TV_ERR_DTYPE, TV_ERR_SHAPE, TV_ERR_TREE,
 * TV_ERR_OVERFLOW, TV_ERR_ALIGN, TV_ERR_CUDA. */
int tv_tree_logits_process(const tv_logits_desc* desc, const void* d_logits, const uint16_t* d_counts,
                           const float* d_penalties, const int32_t* d_bias_offsets, const int32_t* d_bias_tokens,
                           const float* d_bias_values, const uint32_t* d_mask, const int32_t* d_draft_tokens,
                           const int32_t* d_node_offsets, const uint64_t* d_anc, void* d_out, int32_t* d_status,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TREE_LOGITS_H */
