// Parameters of the 4-bit cache's row kernels, resolved on the host.
// Internal to the library.
#pragma once
#include "tv_internal.cuh"

namespace tv {

struct Kv4RowsParams {
  const void* k;             // append: [Hkv, rows, d]
  const void* v;
  void* k_out;               // read: [Hkv, rows, d]
  void* v_out;
  const uint8_t* k4;         // [B, Hkv, max_pages, block] or [num_pages, Hkv, block] (append writes it)
  const uint8_t* v4;
  const int32_t* page_table; // [B, max_pages] or nullptr (contiguous)
  const int32_t* row_offsets;
  const int32_t* start;
  int32_t* status;
  int B, Hkv, d;
  int64_t rows, max_rows, capacity, max_pages, num_pages;
};

struct Kv4CommitParams {
  const int32_t* argmax;
  const int32_t* draft;
  const int32_t* parents;
  const int32_t* node_offsets;
  const void* k_tree;        // [Hkv, R, d]
  const void* v_tree;
  uint8_t* k4;
  uint8_t* v4;
  const int32_t* page_table;
  int32_t* prefix_len;
  int32_t* accept_len;
  int32_t* path;
  int32_t* tokens;
  int32_t* status;
  int B, R, Hkv, d, max_nodes;
  int64_t capacity, max_pages, num_pages;
};

cudaError_t launch_kv4_append(const Kv4RowsParams& p, int dtype, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4RowsParams& p, int dtype, cudaStream_t s);
cudaError_t launch_kv4_commit(const Kv4CommitParams& p, int dtype, cudaStream_t s);

}  // namespace tv
