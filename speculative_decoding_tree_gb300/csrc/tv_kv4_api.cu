// Host side of include/tree_window.h and include/tree_kv4.h: validation,
// launch plans and launches of the windowed attention and of the 4-bit cache.
#include "tree_kv4.h"
#include "tv_host.cuh"
#include "tv_kv4.cuh"
#include "tv_kv4_store.cuh"

namespace tv {
namespace {

constexpr int64_t kNoWindow = (int64_t)1 << 40;     // a window beyond every position

int check_window(const tv_window* w) {
  if (!w) return TV_ERR_NULL;
  return w->window < 1 || w->sinks < 0 ? TV_ERR_SHAPE : TV_OK;
}

// The plan of the windowed and of the 4-bit attention: as make_plan's for the
// CUDA-core and the one-CTA tensor-core kernels, over the keys a call can see
// at most (key_map_bound) instead of max_prefix.
int make_window_plan(const tv_desc* d, const tv_window* w, bool kv4, Plan* p) {
  const int G = d->num_q_heads / d->num_kv_heads;
  // kernel: CUDA cores (0), one tensor-core CTA per row tile (1), and for the
  // 4-bit cache tcgen05 (4) or, for few rows, registers only (5)
  const int warps = simt_warps(d, G);
  int kernel = 0, key_tile = 32, rows_per_tile = warps * (1024 / d->head_dim);
  int ctas_per_sm = simt_ctas_per_sm(d->head_dim, warps);
  int step = 32;                                     // keys a chunk grows by
  if (!kv4 && tc_supported(d, G)) {
    kernel = 1;
    step = key_tile = tc_key_tile(d->head_dim);
    rows_per_tile = (128 / G) * G;
    ctas_per_sm = 1;
  } else if (kv4 && kv4_rows_supported(d, G)) {
    kernel = 5;
    key_tile = kv4_rows_key_tile();
    step = 4 * key_tile;                             // a span for each warp
    rows_per_tile = d->max_nodes * G;
    ctas_per_sm = kv4_rows_ctas_per_sm(d->head_dim);
  } else if (kv4 && kv4_tc_supported(d, G)) {
    kernel = 4;
    step = key_tile = kv4_tc_key_tile();
    const int cols = kv4_tc_columns(d->max_nodes, G, d->head_dim);
    rows_per_tile = cols / G * G;
    ctas_per_sm = kv4_tc_ctas_per_sm(d->head_dim, cols);
  }
  const int row_tiles = (d->max_nodes * G + rows_per_tile - 1) / rows_per_tile;
  p->window = w ? (w->window < kNoWindow ? w->window : kNoWindow) : 0;
  p->sinks = w ? w->sinks : 0;
  p->map_tile = key_tile;
  const int64_t L = key_map_bound(d->max_prefix, p->window, p->sinks, key_tile);
  const int64_t units = (int64_t)d->batch * d->num_kv_heads * row_tiles;
  const int64_t slots = (int64_t)num_sms() * ctas_per_sm;          // CTAs that run at once
  int64_t chunk;
  int tree_tile = 0;
  if (d->batch == 1) {
    // one wave (make_plan's rule); kernel 5 keeps the tree with the last chunk
    int64_t want = slots / units;
    if (want < 1) want = 1;
    const int64_t tiles = (L + step - 1) / step;
    if (tiles > ((int64_t)1 << 30) / step) return TV_ERR_OVERFLOW;
    if (kernel != 5) tree_tile = step;
    int64_t c = (tiles + want - 1) / want;
    if (c < 1) c = 1;
    while (c <= tiles && num_chunks(L, (int)(c * step), tree_tile) > want) ++c;
    chunk = c * step;
  } else {
    // Ragged batch.  Many units: about four waves of CTAs when the sequences
    // are half the longest on average, but no chunk below 1920 keys
    // (make_plan's): 64 sequences x 4 rows 163 us with 1920, 156 with 2816 and
    // 163 with 4096 keys; x 32 rows 315 / 297 / 289; 16 trees of 64 .. 256 rows
    // 177 / 184 / 182.  Few units: chunks that give every CTA slot one, down to
    // 512 keys (4 sequences x 4 rows over 8192 keys 22.0 us, 28.8 with 1920).
    // The CUDA cores' chunks start at 512 keys: their tiles are short
    // (8 trees of 40 .. 120 rows over up to 2500 keys 645 us, 980 with 1920).
    const double wave = (double)units * L / slots, even = wave / 8;
    const double least = kernel == 0 ? 512 : (wave < 512 ? 512 : (wave < 1920 ? wave : 1920));
    chunk = align_up((int64_t)(even < least ? least : (even > 8192 ? 8192 : even)), step);
  }
  if (chunk > (int64_t)1 << 30) return TV_ERR_OVERFLOW;
  const int splits = num_chunks(L, (int)chunk, tree_tile);
  const int64_t grid = units * splits;
  if (grid > ((int64_t)1 << 31) - 1) return TV_ERR_OVERFLOW;
  // grids: sequences on z, (KV head, split) or, kernel 0, splits on y, the merge's (KV head, row tile) on y
  const int64_t grid_y = kernel ? (int64_t)d->num_kv_heads * splits : (int64_t)splits;
  if (d->batch > kMaxGridYZ || (int64_t)d->num_kv_heads * row_tiles > kMaxGridYZ || grid_y > kMaxGridYZ)
    return TV_ERR_SHAPE;
  p->G = G;
  p->tree_tile = tree_tile;
  p->pub.kernel = kernel;
  p->pub.num_splits = splits;
  p->pub.chunk = (int)chunk;
  p->pub.row_tiles = row_tiles;
  p->pub.rows_per_tile = rows_per_tile;
  p->pub.grid_ctas = (int)grid;
  p->counter_bytes = 0;
  p->tile_stride = kernel == 1 ? 128 : rows_per_tile;
  int64_t t, o_bytes, ml_bytes;
  if (!mul_ok(splits, d->batch, &t) || !mul_ok(t, d->num_kv_heads, &t) || !mul_ok(t, row_tiles, &t) ||
      !mul_ok(t, p->tile_stride, &t))
    return TV_ERR_OVERFLOW;
  if (!mul_ok(t, (int64_t)d->head_dim * (part_bf16(d, *p) ? 2 : 4), &o_bytes) || !mul_ok(t, 8, &ml_bytes))
    return TV_ERR_OVERFLOW;
  p->o_part_bytes = align_up(o_bytes, 256);
  p->ml_part_bytes = align_up(ml_bytes, 256);
  return TV_OK;
}

int validate_kv4(const tv_desc* d) {
  const int rc = validate(d);
  if (rc) return rc;
  return d->capacity % kPageSize ? TV_ERR_SHAPE : TV_OK;
}

// The descriptor of calls on the cache alone: it has no tree, so max_nodes and
// total_rows may hold anything.
int validate_cache(const tv_desc* d) {
  if (!d) return TV_ERR_NULL;
  tv_desc c = *d;
  c.max_nodes = 1;
  c.total_rows = c.batch;
  return validate_kv4(&c);
}

int plan_of(const tv_desc* d, const tv_window* w, bool kv4, Plan* p) {
  int rc = kv4 ? validate_kv4(d) : validate(d);
  if (rc) return rc;
  if (!kv4 || w) {
    rc = check_window(w);
    if (rc) return rc;
  }
  return make_window_plan(d, w, kv4, p);
}

int workspace_of(const tv_desc* d, const tv_window* w, bool kv4, size_t* bytes) {
  Plan p;
  const int rc = plan_of(d, w, kv4, &p);
  if (rc) return rc;
  if (!bytes) return TV_ERR_NULL;
  *bytes = (size_t)p.part_bytes();
  return TV_OK;
}

int public_plan_of(const tv_desc* d, const tv_window* w, bool kv4, tv_plan* plan) {
  Plan p;
  const int rc = plan_of(d, w, kv4, &p);
  if (rc) return rc;
  if (!plan) return TV_ERR_NULL;
  *plan = p.pub;
  return TV_OK;
}

int attention(const tv_desc* d, const tv_window* w, bool kv4, const void* q, const void* kc, const void* vc,
              const int32_t* pt, const int32_t* plen, const int32_t* no, const void* kt, const void* vt,
              const uint64_t* anc, const int32_t* depth, void* out, void* ws, size_t ws_bytes, int32_t* st,
              void* stream) {
  Plan p;
  int rc = plan_of(d, w, kv4, &p);
  if (rc) return rc;
  rc = check_attn_ptrs(d, q, kc, vc, pt, plen, no, kt, vt, anc, ws, st);
  if (rc) return rc;
  if (!out || (w && !depth)) return TV_ERR_NULL;
  if (!aligned16(out) || (depth && !aligned16(depth))) return TV_ERR_ALIGN;
  if ((int64_t)ws_bytes < p.part_bytes()) return TV_ERR_WORKSPACE;
  AttnParams a = attn_params(d, p, q, kc, vc, pt, plen, no, kt, vt, anc, ws, st);
  a.depth = depth;
  a.out = out;                                       // one-chunk sequences are finished by the split pass
  const cudaStream_t s = as_stream(stream);
  const cudaError_t e = p.pub.kernel == 5   ? launch_attn_kv4_rows(a, s)
                        : p.pub.kernel == 4 ? launch_attn_kv4(a, kv4_tc_columns(d->max_nodes, p.G, d->head_dim), s)
                        : kv4               ? launch_attn_simt_kv4(a, d->dtype, s)
                        : p.pub.kernel == 1 ? launch_attn_tc_window(a, s)
                                            : launch_attn_simt_window(a, d->dtype, s);
  if (e != cudaSuccess) return TV_ERR_CUDA;
  if (p.pub.num_splits == 1) return TV_OK;
  return launch_merge_from(d, p, plen, no, out, ws, st, s, 1);
}

// validation and parameters shared by append and read
int rows_params(const tv_desc* d, int64_t rows, int64_t max_rows, const void* k, const void* v,
                const int32_t* offs, const int32_t* start, const void* k4, const void* v4, const int32_t* pt,
                int32_t* st, Kv4RowsParams* p) {
  const int rc = validate_cache(d);
  if (rc) return rc;
  if (rows < 0 || max_rows < 0 || rows > ((int64_t)1 << 31) - 1) return TV_ERR_SHAPE;
  const bool some = rows > 0 && max_rows > 0;
  if ((some && (!k || !v)) || !offs || !start || !k4 || !v4 || !st) return TV_ERR_NULL;
  if (d->page_size == kPageSize && !pt) return TV_ERR_NULL;
  const void* all[] = {k, v, offs, start, k4, v4, st};
  for (const void* x : all)
    if (!aligned16(x)) return TV_ERR_ALIGN;
  if (pt && !aligned16(pt)) return TV_ERR_ALIGN;
  if (d->batch > kMaxGridYZ || d->num_kv_heads > kMaxGridYZ) return TV_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(rows, d->num_kv_heads, &t) || !mul_ok(t, (int64_t)d->head_dim * 4, &t)) return TV_ERR_OVERFLOW;
  *p = Kv4RowsParams{};
  p->k4 = reinterpret_cast<const uint8_t*>(k4);
  p->v4 = reinterpret_cast<const uint8_t*>(v4);
  p->page_table = d->page_size ? pt : nullptr;
  p->row_offsets = offs;
  p->start = start;
  p->status = st;
  p->B = d->batch; p->Hkv = d->num_kv_heads; p->d = d->head_dim;
  p->rows = rows;
  p->max_rows = max_rows < rows ? max_rows : rows;
  p->capacity = d->capacity;
  p->max_pages = d->capacity / kPageSize;
  p->num_pages = d->num_pages;
  return TV_OK;
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_window_workspace_size(const tv_desc* desc, const tv_window* win, size_t* bytes) {
  return workspace_of(desc, win, false, bytes);
}

int tv_window_attn_plan(const tv_desc* desc, const tv_window* win, tv_plan* plan) {
  return public_plan_of(desc, win, false, plan);
}

int tree_verify_attn_window(const tv_desc* desc, const tv_window* win, const void* d_q, const void* d_k_cache,
                            const void* d_v_cache, const int32_t* d_page_table, const int32_t* d_prefix_len,
                            const int32_t* d_node_offsets, const void* d_k_tree, const void* d_v_tree,
                            const uint64_t* d_anc, const int32_t* d_depth, void* d_out, void* d_workspace,
                            size_t workspace_bytes, int32_t* d_status, void* stream) {
  return attention(desc, win, false, d_q, d_k_cache, d_v_cache, d_page_table, d_prefix_len, d_node_offsets, d_k_tree,
                   d_v_tree, d_anc, d_depth, d_out, d_workspace, workspace_bytes, d_status, stream);
}

int tv_kv4_cache_bytes(const tv_desc* desc, int64_t* k_bytes, int64_t* v_bytes) {
  const int rc = validate_cache(desc);
  if (rc) return rc;
  if (!k_bytes || !v_bytes) return TV_ERR_NULL;
  // below the fp32/bf16 cache's size, which validate() checked against int64
  const int64_t blocks = (desc->page_size ? desc->num_pages : desc->batch * (desc->capacity / kPageSize)) *
                         desc->num_kv_heads;
  *k_bytes = blocks * kv4::k_block_bytes(desc->head_dim);
  *v_bytes = blocks * kv4::v_block_bytes(desc->head_dim);
  return TV_OK;
}

int tv_kv4_append(const tv_desc* desc, int64_t rows, int64_t max_rows, const void* d_k, const void* d_v,
                  const int32_t* d_row_offsets, const int32_t* d_start, void* d_k4, void* d_v4,
                  const int32_t* d_page_table, int32_t* d_status, void* stream) {
  Kv4RowsParams p;
  const int rc = rows_params(desc, rows, max_rows, d_k, d_v, d_row_offsets, d_start, d_k4, d_v4, d_page_table,
                             d_status, &p);
  if (rc) return rc;
  if (p.max_rows == 0) return TV_OK;
  p.k = d_k;
  p.v = d_v;
  return launch_kv4_append(p, desc->dtype, as_stream(stream)) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

int tv_kv4_read(const tv_desc* desc, int64_t rows, int64_t max_rows, const void* d_k4, const void* d_v4,
                const int32_t* d_page_table, const int32_t* d_row_offsets, const int32_t* d_start, void* d_k,
                void* d_v, int32_t* d_status, void* stream) {
  Kv4RowsParams p;
  const int rc = rows_params(desc, rows, max_rows, d_k, d_v, d_row_offsets, d_start, d_k4, d_v4, d_page_table,
                             d_status, &p);
  if (rc) return rc;
  if (p.max_rows == 0) return TV_OK;
  p.k_out = d_k;
  p.v_out = d_v;
  return launch_kv4_read(p, desc->dtype, as_stream(stream)) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

int tree_accept_commit_argmax_kv4(const tv_desc* desc, const int32_t* d_argmax, const int32_t* d_draft_tokens,
                                  const int32_t* d_parents, const int32_t* d_node_offsets, const void* d_k_tree,
                                  const void* d_v_tree, void* d_k4, void* d_v4, const int32_t* d_page_table,
                                  int32_t* d_prefix_len, int32_t* d_accept_len, int32_t* d_path, int32_t* d_tokens,
                                  int32_t* d_status, void* stream) {
  const int rc = validate_kv4(desc);
  if (rc) return rc;
  if (desc->batch > kMaxGridYZ) return TV_ERR_SHAPE;
  if (!d_argmax || !d_draft_tokens || !d_parents || !d_node_offsets || !d_k_tree || !d_v_tree || !d_k4 || !d_v4 ||
      !d_prefix_len || !d_accept_len || !d_path || !d_tokens || !d_status)
    return TV_ERR_NULL;
  if (desc->page_size == kPageSize && !d_page_table) return TV_ERR_NULL;
  const void* all[] = {d_argmax, d_draft_tokens, d_parents, d_node_offsets, d_k_tree, d_v_tree, d_k4,
                       d_v4, d_prefix_len, d_accept_len, d_path, d_tokens, d_status};
  for (const void* x : all)
    if (!aligned16(x)) return TV_ERR_ALIGN;
  if (d_page_table && !aligned16(d_page_table)) return TV_ERR_ALIGN;
  Kv4CommitParams p = {};
  p.argmax = d_argmax; p.draft = d_draft_tokens; p.parents = d_parents; p.node_offsets = d_node_offsets;
  p.k_tree = d_k_tree; p.v_tree = d_v_tree;
  p.k4 = reinterpret_cast<uint8_t*>(d_k4); p.v4 = reinterpret_cast<uint8_t*>(d_v4);
  p.page_table = desc->page_size ? d_page_table : nullptr;
  p.prefix_len = d_prefix_len; p.accept_len = d_accept_len; p.path = d_path; p.tokens = d_tokens;
  p.status = d_status;
  p.B = desc->batch; p.R = desc->total_rows; p.Hkv = desc->num_kv_heads; p.d = desc->head_dim;
  p.max_nodes = desc->max_nodes; p.capacity = desc->capacity; p.max_pages = desc->capacity / kPageSize;
  p.num_pages = desc->num_pages;
  return launch_kv4_commit(p, desc->dtype, as_stream(stream)) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

int tv_kv4_workspace_size(const tv_desc* desc, const tv_window* win, size_t* bytes) {
  return workspace_of(desc, win, true, bytes);
}

int tv_kv4_attn_plan(const tv_desc* desc, const tv_window* win, tv_plan* plan) {
  return public_plan_of(desc, win, true, plan);
}

int tree_verify_attn_kv4(const tv_desc* desc, const tv_window* win, const void* d_q, const void* d_k4,
                         const void* d_v4, const int32_t* d_page_table, const int32_t* d_prefix_len,
                         const int32_t* d_node_offsets, const void* d_k_tree, const void* d_v_tree,
                         const uint64_t* d_anc, const int32_t* d_depth, void* d_out, void* d_workspace,
                         size_t workspace_bytes, int32_t* d_status, void* stream) {
  return attention(desc, win, true, d_q, d_k4, d_v4, d_page_table, d_prefix_len, d_node_offsets, d_k_tree, d_v_tree,
                   d_anc, d_depth, d_out, d_workspace, workspace_bytes, d_status, stream);
}

}  // extern "C"
