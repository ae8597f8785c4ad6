// What the prompt attention's kernels share: parameters, the keys' tiles, the
// work units of a ragged batch and the partials of a split.  Internal.
//
// Keys of a sequence are counted in tiles of 128: the prefix's tiles first
// (Pt = ceil(P / 128), the last one partly empty), then the rows' own.  Row i
// sees tiles 0 .. Pt + i / 128.  A split s takes the tiles [s ct, (s + 1) ct);
// row i has (Pt + i / 128) / ct + 1 of them, and a row with one is written by
// its own CTA, the others by the merge from fp32 partials.
//
// A unit is `rows_per_unit` query rows (token, group head) of one sequence and
// KV head.  Units are numbered by sequence, within one from its last rows (the
// most keys) down: CTAs that run at the same time then read the same keys
// from L2, and a sequence's tail is short work.  (Numbered by level over all
// sequences, the 16 prompts of the batch read 531 MB from memory instead of
// 265 and took 389 us instead of 369.)
#pragma once

#include "tree_prompt.h"
#include "tv_internal.cuh"

namespace tv {

constexpr int kPromptTile = 128;

struct PromptParams {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* page_table;
  const int32_t* prefix_len;
  const int32_t* row_offsets;
  const void* k_rows;
  const void* v_rows;
  void* out;
  float* o_part;             // [rows, Hq, splits, d] O_s / l_s of rows with two splits or more
  float2* ml_part;           // [rows, Hq, splits] running maximum (log2 units) and sum
  void* split;               // fp32: the numbers in three bf16 parts, in blocks
  int32_t* status;
  int B, Hq, Hkv, G, d, paged, out_bf16;
  int rows_per_tile;         // query rows of a 128-row tile in use (tensor cores: a multiple of G)
  int rows_per_unit;
  int unit_tokens;           // rows_per_unit / G where G divides it (tensor-core tiles of bf16), else 0
  int chunk_tiles, splits;   // ct, and the grid's splits
  int64_t rows, max_rows;
  int64_t capacity, num_pages, max_pages, max_prefix;
  float scale_log2;
};

// Rows of sequence b; false (and TV_DEV_BAD_OFFSETS) when they are no valid range.
__device__ inline bool prompt_rows(const int32_t* offs, int b, int64_t rows, int64_t max_rows, int32_t* status,
                                   int64_t* o0, int64_t* n) {
  const int64_t a = offs[b], c = offs[b + 1];
  if (a < 0 || c < a || c > rows || c - a > max_rows || (b == 0 && a != 0)) {
    set_status(status, TV_DEV_BAD_OFFSETS);
    *o0 = *n = 0;
    return false;
  }
  *o0 = a;
  *n = c - a;
  return true;
}

// Upper bound of the units of all sequences (one KV head).
inline int64_t prompt_units(int64_t rows, int64_t max_rows, int B, int G, int rows_per_unit) {
  const int64_t packed = rows * G / rows_per_unit + B;
  const int64_t padded = ((max_rows * G + rows_per_unit - 1) / rows_per_unit) * B;
  return packed < padded ? packed : padded;
}

// What a CTA works on: unit i of sequence b (-1: nothing), whose rows are
// o0 .. o0 + n - 1 behind P cached positions.
struct PromptUnit {
  int b, i, o0, n;
  int64_t P;
};

// Whole warp: unit u of the numbering above, left in *out.
__device__ inline void find_unit(const PromptParams& p, unsigned u, PromptUnit* out) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int64_t raw = b < p.B ? p.prefix_len[b] : 0;
    int64_t o0 = 0, n = 0;
    if (b < p.B) prompt_rows(p.row_offsets, b, p.rows, p.max_rows, p.status, &o0, &n);
    const unsigned mine = p.unit_tokens > 0 ? ((unsigned)n + p.unit_tokens - 1) / (unsigned)p.unit_tokens
                                            : (unsigned)((n * p.G + p.rows_per_unit - 1) / p.rows_per_unit);
    unsigned end = mine;                            // units of these sequences up to this lane's
    if (p.B > 1) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned v = __shfl_up_sync(kAll, end, d);
        if (lane >= d) end += v;
      }
    }
    const unsigned hit = __ballot_sync(kAll, u < end && u >= end - mine);
    if (hit) {
      if (hit >> lane & 1u) {
        const int64_t P = clamp_prefix(raw, p.max_prefix, p.capacity);
        if (P != raw) set_status(p.status, TV_DEV_BAD_PREFIX);
        *out = PromptUnit{b, (int)(end - 1 - u), (int)o0, (int)n, P};
      }
      return;
    }
    u -= __shfl_sync(kAll, end, p.B > 1 ? 31 : 0);
  }
  if (lane == 0) *out = PromptUnit{-1, 0, 0, 0, 0};   // no rows, no tiles
}

__host__ __device__ inline int64_t prompt_slot(int64_t row, int h, int s, int Hq, int splits) {
  return (row * Hq + h) * splits + s;
}

int validate_prompt(const tv_desc* d, int64_t rows, int64_t max_rows);
cudaError_t launch_prompt_merge(const PromptParams& p, cudaStream_t s);
bool prompt_tc_supported(const tv_desc* d, int64_t rows);   // the tensor-core kernels' tiles fit the call
cudaError_t launch_prompt_tc(const PromptParams& p, int64_t units, cudaStream_t s);
int64_t prompt_f32_bytes(const tv_desc* d, int64_t rows);   // of the blocks; -1: more than a call can have
cudaError_t launch_prompt_f32(const PromptParams& p, int dtype, int64_t units, cudaStream_t s);
cudaError_t launch_prompt_tc2(const PromptParams& p, int64_t units, cudaStream_t s);

}  // namespace tv
