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

// Whole warp: unit u of the numbering above, left in *out.  f(L) = units at
// level L or above, over all sequences; u's level is the largest L with
// f(L) > u.  A lane keeps its first sequence (of up to 32) in registers.  Of
// one sequence the level is known without a search (1200 clocks of a CTA).
__device__ inline void find_unit(const PromptParams& p, unsigned u, PromptUnit* out) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto units = [&](int64_t n) -> unsigned {
    if (p.unit_tokens > 0) return ((unsigned)n + p.unit_tokens - 1) / (unsigned)p.unit_tokens;
    return (unsigned)((n * p.G + p.rows_per_unit - 1) / p.rows_per_unit);
  };
  auto load = [&](int b, int64_t* o0, int64_t* n) {
    *o0 = *n = 0;
    if (b < p.B) prompt_rows(p.row_offsets, b, p.rows, p.max_rows, p.status, o0, n);
  };
  const int64_t raw0 = lane < p.B ? p.prefix_len[lane] : 0;
  int64_t o0, n0;
  load(lane, &o0, &n0);
  const unsigned has = units(n0);
  auto each_later = [&](auto f) {                   // the units of sequences past the first 32
    for (int b = lane + 32; b < p.B; b += 32) {
      int64_t x, m;
      load(b, &x, &m);
      f(units(m));
    }
  };
  auto at_or_above = [&](unsigned L) -> unsigned {
    unsigned v = has > L ? has - L : 0u;
    each_later([&](unsigned t) { v += t > L ? t - L : 0u; });
    return __reduce_add_sync(kAll, v);
  };
  auto put = [&](int b, unsigned i, int64_t a, int64_t m, int64_t raw) {
    const int64_t c = clamp_prefix(raw, p.max_prefix, p.capacity);
    if (c != raw) set_status(p.status, TV_DEV_BAD_PREFIX);
    *out = PromptUnit{b, (int)i, (int)a, (int)m, c};
  };
  if (p.B == 1) {
    if (lane == 0) {
      if (u < has) put(0, has - 1 - u, o0, n0, raw0);
      else *out = PromptUnit{-1, 0, 0, 0, 0};
    }
    return;
  }
  if (at_or_above(0) <= u) {
    if (lane == 0) *out = PromptUnit{-1, 0, 0, 0, 0};   // no rows, no tiles
    return;
  }
  unsigned top = has, lo = 0;
  each_later([&](unsigned t) { top = max(top, t); });
  unsigned hi = __reduce_max_sync(kAll, top);       // f(hi) = 0
  while (hi - lo > 1) {
    const unsigned mid = (lo + hi) >> 1;
    if (at_or_above(mid) > u) lo = mid;
    else hi = mid;
  }
  unsigned rank = u - at_or_above(lo + 1);          // among the sequences with a unit at this level
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int64_t a = o0, m = n0;
    if (b0 > 0) load(b, &a, &m);
    const unsigned w = __ballot_sync(kAll, units(m) > lo);
    if (rank < (unsigned)__popc(w)) {
      if ((w >> lane & 1u) && (unsigned)__popc(w & ((1u << lane) - 1)) == rank)
        put(b, lo, a, m, b0 > 0 ? (int64_t)p.prefix_len[b] : raw0);
      return;
    }
    rank -= __popc(w);
  }
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
