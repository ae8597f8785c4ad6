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
// KV head.  Units are numbered from the longest rows down (by their place in
// the sequence, over all sequences), so the grid's tail is short work.
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

// Whole warp: unit u of the numbering above as (sequence, index of the unit in
// it); false past the last.  f(L) = units at level L or above, over all
// sequences; u's level is the largest L with f(L) > u.
__device__ inline bool find_unit(const PromptParams& p, int64_t u, int* b_out, int* i_out) {
  const int lane = threadIdx.x & 31;
  auto tiles = [&](int b) -> int64_t {
    if (b >= p.B) return 0;
    int64_t o0, n;
    prompt_rows(p.row_offsets, b, p.rows, p.max_rows, p.status, &o0, &n);
    return (n * p.G + p.rows_per_unit - 1) / p.rows_per_unit;
  };
  auto sum = [](int64_t v) {
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
  };
  const int64_t mine = tiles(lane);                 // of the first 32 sequences, kept in a register
  auto at_or_above = [&](int64_t L) -> int64_t {
    int64_t v = mine > L ? mine - L : 0;
    for (int b = lane + 32; b < p.B; b += 32) {
      const int64_t t = tiles(b);
      if (t > L) v += t - L;
    }
    return sum(v);
  };
  if (at_or_above(0) <= u) return false;
  int64_t lo = 0, hi = (p.max_rows * p.G + p.rows_per_unit - 1) / p.rows_per_unit;   // f(lo) > u, f(hi) = 0
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (at_or_above(mid) > u) lo = mid;
    else hi = mid;
  }
  int64_t rank = u - at_or_above(lo + 1);           // among the sequences with a unit at this level
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const bool has = (b0 == 0 ? mine : tiles(b0 + lane)) > lo;
    const unsigned m = __ballot_sync(0xffffffffu, has);
    if (rank < __popc(m)) {
      const bool me = has && __popc(m & ((1u << lane) - 1)) == rank;
      *b_out = b0 + __ffs(__ballot_sync(0xffffffffu, me)) - 1;
      *i_out = (int)lo;
      return true;
    }
    rank -= __popc(m);
  }
  return false;
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
