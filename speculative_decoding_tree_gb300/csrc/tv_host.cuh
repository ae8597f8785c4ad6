// Host-side pieces the C ABI's translation units share: checked arithmetic,
// descriptor validation, the launch plan, the attention's parameter block and
// the merge.  Internal to the library.
#pragma once

#include <stddef.h>

#include "tv_internal.cuh"

namespace tv {

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
inline bool add_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_add_overflow(a, b, out); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

cudaStream_t as_stream(void* s);

struct Plan {
  tv_plan pub;
  int G;
  int tree_tile;             // num_chunks rule: 0, or the key tile (one-wave plans)
  int tile_stride;
  int64_t o_part_bytes, ml_part_bytes;
  int64_t counter_bytes;     // the persistent kernel's work counter (0 for the other kernels)
  int64_t window = 0, sinks = 0;   // key_map (window 0: the whole prefix)
  int map_tile = 1;
  int64_t part_bytes() const { return o_part_bytes + ml_part_bytes + counter_bytes; }
};

int validate(const tv_desc* d);

int check_attn_ptrs(const tv_desc* d, const void* q, const void* kc, const void* vc, const int32_t* pt,
                    const int32_t* pl, const int32_t* no, const void* kt, const void* vt, const uint64_t* anc,
                    const void* ws, int32_t* st);

int part_bf16(const tv_desc* d, const Plan& pl);

AttnParams attn_params(const tv_desc* d, const Plan& pl, const void* q, const void* kc, const void* vc,
                       const int32_t* pt, const int32_t* plen, const int32_t* no, const void* kt, const void* vt,
                       const uint64_t* anc, void* ws, int32_t* st);

int launch_merge_from(const tv_desc* d, const Plan& pl, const int32_t* plen, const int32_t* no, void* out,
                      const void* ws, int32_t* st, cudaStream_t s, int skip_single);

}  // namespace tv
