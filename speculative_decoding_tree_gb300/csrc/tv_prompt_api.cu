// Host side of include/tree_prompt.h: validation, the launch plan and the
// launches of the prompt attention.
#include <cmath>

#include "tv_host.cuh"
#include "tv_prompt.cuh"

namespace tv {
namespace {

struct PromptPlan {
  tv_plan pub;
  int64_t units;             // per KV head
  int rows_per_unit;
  int64_t o_bytes, ml_bytes, split_bytes;
};

}  // namespace

// The descriptor without its tree, which these calls do not have.
int validate_prompt(const tv_desc* d, int64_t rows, int64_t max_rows) {
  if (!d) return TV_ERR_NULL;
  tv_desc c = *d;
  c.max_nodes = 1;
  c.total_rows = c.batch;
  const int rc = validate(&c);
  if (rc) return rc;
  if (rows < 0 || max_rows < 0 || rows > ((int64_t)1 << 31) - 1) return TV_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(rows, d->num_q_heads, &t) || !mul_ok(t, (int64_t)d->head_dim * 4, &t)) return TV_ERR_OVERFLOW;
  return TV_OK;
}

namespace {

int make_prompt_plan(const tv_desc* d, int64_t rows, int64_t max_rows, PromptPlan* p) {
  const int G = d->num_q_heads / d->num_kv_heads;
  if (max_rows > rows) max_rows = rows;
  p->pub = tv_plan{};
  p->pub.kernel = prompt_tc_supported(d, rows) ? (d->head_dim == 128 ? 6 : 7) : 8;
  const bool parts = p->pub.kernel == 8;             // numbers in three parts: one query tile a unit, any grouping
  p->pub.rows_per_tile = parts ? 128 : 128 / G * G;
  p->rows_per_unit = parts ? 128 : 2 * p->pub.rows_per_tile;
  p->units = prompt_units(rows, max_rows, d->batch, G, p->rows_per_unit);
  const int64_t tiles = (d->max_prefix + kPromptTile - 1) / kPromptTile + (max_rows + kPromptTile - 1) / kPromptTile;
  // Few units of many keys are split over the keys: so that about every SM has
  // one, in chunks of four tiles or more; kernel 8, whose tiles take longer,
  // into about two waves of chunks of any length (2000 fp32 rows x 4 heads at
  // head_dim 256: 134, 84, 113 and 101 us with 1, 2, 3 and 4).
  const int64_t sms = num_sms();
  int64_t ctas;
  if (!mul_ok(p->units, d->num_kv_heads, &ctas) || !mul_ok(ctas, p->pub.kernel == 6 ? 1 : d->head_dim / 128, &ctas))
    return TV_ERR_OVERFLOW;
  int64_t want = ctas > 0 ? (parts ? 2 * sms : sms) / ctas : 1;
  if (!parts && want > tiles / 4) want = tiles / 4;
  if (want > tiles) want = tiles;
  if (want < 1) want = 1;
  const int64_t chunk = tiles > 0 ? (tiles + want - 1) / want : 1;
  const int64_t splits = tiles > 0 ? (tiles + chunk - 1) / chunk : 1;
  if (chunk > ((int64_t)1 << 30) / kPromptTile) return TV_ERR_OVERFLOW;
  int64_t grid;
  if (!mul_ok(ctas, splits, &grid) || grid > ((int64_t)1 << 31) - 1) return TV_ERR_OVERFLOW;
  p->pub.chunk = (int)(chunk * kPromptTile);
  p->pub.num_splits = (int)splits;
  p->pub.row_tiles = (int)((max_rows * G + p->pub.rows_per_tile - 1) / p->pub.rows_per_tile);
  p->pub.grid_ctas = (int)grid;
  p->o_bytes = p->ml_bytes = p->split_bytes = 0;
  if (parts) {
    p->split_bytes = prompt_f32_bytes(d, rows);
    if (p->split_bytes < 0) return TV_ERR_OVERFLOW;
  }
  if (splits > 1) {
    int64_t t;
    if (!mul_ok(rows, d->num_q_heads, &t) || !mul_ok(t, splits, &t) || !mul_ok(t, 8, &p->ml_bytes) ||
        !mul_ok(t, (int64_t)d->head_dim * 4, &p->o_bytes))
      return TV_ERR_OVERFLOW;
    if ((rows * d->num_q_heads + 7) / 8 > ((int64_t)1 << 31) - 1) return TV_ERR_OVERFLOW;   // the merge's grid
    if (p->split_bytes > ((int64_t)1 << 62) - p->o_bytes || p->o_bytes > (int64_t)1 << 61) return TV_ERR_OVERFLOW;
    p->o_bytes = align_up(p->o_bytes, 256);
    p->ml_bytes = align_up(p->ml_bytes, 256);
  }
  return TV_OK;
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_prompt_workspace_size(const tv_desc* desc, int64_t rows, int64_t max_rows, size_t* bytes) {
  int rc = validate_prompt(desc, rows, max_rows);
  if (rc) return rc;
  if (!bytes) return TV_ERR_NULL;
  PromptPlan p;
  rc = make_prompt_plan(desc, rows, max_rows, &p);
  if (rc) return rc;
  *bytes = (size_t)(p.o_bytes + p.ml_bytes + p.split_bytes);
  return TV_OK;
}

int tv_prompt_attn_plan(const tv_desc* desc, int64_t rows, int64_t max_rows, tv_plan* plan) {
  int rc = validate_prompt(desc, rows, max_rows);
  if (rc) return rc;
  if (!plan) return TV_ERR_NULL;
  PromptPlan p;
  rc = make_prompt_plan(desc, rows, max_rows, &p);
  if (rc) return rc;
  *plan = p.pub;
  return TV_OK;
}

int tv_prompt_attn(const tv_desc* desc, int64_t rows, int64_t max_rows, const void* d_q, const void* d_k_cache,
                   const void* d_v_cache, const int32_t* d_page_table, const int32_t* d_prefix_len,
                   const int32_t* d_row_offsets, const void* d_k_rows, const void* d_v_rows, void* d_out,
                   void* d_workspace, size_t workspace_bytes, int32_t* d_status, void* stream) {
  int rc = validate_prompt(desc, rows, max_rows);
  if (rc) return rc;
  PromptPlan pl;
  rc = make_prompt_plan(desc, rows, max_rows, &pl);
  if (rc) return rc;
  if (rows == 0 || max_rows == 0) return TV_OK;
  const bool split = pl.pub.num_splits > 1, cache = desc->max_prefix > 0;
  if (!d_q || !d_prefix_len || !d_row_offsets || !d_k_rows || !d_v_rows || !d_out || !d_status ||
      ((split || pl.split_bytes) && !d_workspace) || (cache && (!d_k_cache || !d_v_cache)) ||
      (cache && desc->page_size == kPageSize && !d_page_table))
    return TV_ERR_NULL;
  const void* all[] = {d_q,      d_k_cache, d_v_cache,   d_page_table, d_prefix_len, d_row_offsets,
                       d_k_rows, d_v_rows,  d_workspace, d_out,        d_status};
  for (const void* x : all)
    if (!aligned16(x)) return TV_ERR_ALIGN;
  if ((int64_t)workspace_bytes < pl.o_bytes + pl.ml_bytes + pl.split_bytes) return TV_ERR_WORKSPACE;
  PromptParams p = {};
  p.q = d_q; p.k_cache = d_k_cache; p.v_cache = d_v_cache;
  p.page_table = desc->page_size ? d_page_table : nullptr;
  p.prefix_len = d_prefix_len; p.row_offsets = d_row_offsets; p.k_rows = d_k_rows; p.v_rows = d_v_rows;
  p.out = d_out;
  p.o_part = reinterpret_cast<float*>(d_workspace);
  p.ml_part = reinterpret_cast<float2*>(reinterpret_cast<char*>(d_workspace) + pl.o_bytes);
  p.split = reinterpret_cast<char*>(d_workspace) + pl.o_bytes + pl.ml_bytes;
  p.status = d_status;
  p.B = desc->batch; p.Hq = desc->num_q_heads; p.Hkv = desc->num_kv_heads; p.G = p.Hq / p.Hkv;
  p.d = desc->head_dim;
  p.paged = desc->page_size != 0;
  p.out_bf16 = desc->dtype == TV_BF16 && !desc->out_f32;
  p.rows_per_tile = pl.pub.rows_per_tile;
  p.rows_per_unit = pl.rows_per_unit;
  p.unit_tokens = pl.pub.kernel == 8 ? 0 : pl.rows_per_unit / p.G;
  p.chunk_tiles = pl.pub.chunk / kPromptTile;
  p.splits = pl.pub.num_splits;
  p.rows = rows;
  p.max_rows = max_rows < rows ? max_rows : rows;
  p.capacity = desc->capacity; p.num_pages = desc->num_pages; p.max_pages = desc->capacity / kPageSize;
  p.max_prefix = desc->max_prefix;
  const float scale = desc->scale > 0.f ? desc->scale : 1.0f / std::sqrt((float)desc->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  const cudaStream_t s = as_stream(stream);
  cudaError_t e = pl.pub.kernel == 8   ? launch_prompt_f32(p, desc->dtype, pl.units, s)
                  : pl.pub.kernel == 7 ? launch_prompt_tc2(p, pl.units, s)
                                       : launch_prompt_tc(p, pl.units, s);
  if (e == cudaSuccess && split) e = launch_prompt_merge(p, s);
  return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // extern "C"
