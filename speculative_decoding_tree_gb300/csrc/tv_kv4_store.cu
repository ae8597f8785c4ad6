// Writing and reading the 4-bit cache (include/tree_kv4.h): rows in, the
// accepted path of a verify step in, rows out.
//
// Quantisation of a group with largest magnitude A (32 channels of K, all
// channels of V at one position): the smallest scale s with 7 s >= A, then
// q = round(x / s) to even, |q| <= 7, u = q + 8.  The quotient is taken with
// a reciprocal and corrected by the exact residual x - q s (one fused
// multiply-add: it has no more bits than x), so the result is that of exact
// arithmetic, ties included.
//
// One CTA handles the 16-position block of one KV head, K and V.  K is
// quantised where it is loaded: four lanes hold a position's 32-channel group
// and share its maximum.  V's codes run along the positions, so its 16 rows
// are staged in shared memory once and read back by channel; a block that is
// written in part keeps the other positions' nibbles.  Both directions are
// bound by the bytes they move; nothing is read twice.
#include "tv_kv4.cuh"
#include "tv_kv4_store.cuh"

namespace tv {
namespace {

using namespace kv4;

constexpr int kThreads = 128;

// 8 values of a row in global memory (through L2: rows are read once)
template <typename T>
__device__ __forceinline__ void load_row8(const T* src, float (&x)[8]);

template <>
__device__ __forceinline__ void load_row8<float>(const float* src, float (&x)[8]) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(src)), b = __ldcg(reinterpret_cast<const float4*>(src) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <>
__device__ __forceinline__ void load_row8<__nv_bfloat16>(const __nv_bfloat16* src, float (&x)[8]) {
  const uint4 u = __ldcg(reinterpret_cast<const uint4*>(src));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    x[2 * t] = __uint_as_float(w[t] << 16);
    x[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
  }
}

__device__ __forceinline__ void store_row8(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store_row8(__nv_bfloat16* dst, const float (&x)[8]) {
  uint4 u;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) h[t] = __floats2bfloat162_rn(x[2 * t], x[2 * t + 1]);   // exact: 7 significant bits
  u.x = *reinterpret_cast<uint32_t*>(&h[0]);
  u.y = *reinterpret_cast<uint32_t*>(&h[1]);
  u.z = *reinterpret_cast<uint32_t*>(&h[2]);
  u.w = *reinterpret_cast<uint32_t*>(&h[3]);
  *reinterpret_cast<uint4*>(dst) = u;
}

__device__ __forceinline__ float no_nan(float x) { return x != x ? 0.f : x; }

// smallest code whose 7 steps reach amax (255 if none): a guess from amax / 7
// in rounded arithmetic, then stepped to the exact answer (7 s is exact)
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const int bits = __float_as_int(amax * (1.f / 7.f));
  int c = (bits - (112 << 23)) >> 20;
  c = c < 0 ? 0 : (c > 255 ? 255 : c);
  while (c < 255 && 7.f * scale_of((uint32_t)c) < amax) ++c;
  while (c > 0 && 7.f * scale_of((uint32_t)c - 1) >= amax) --c;
  return (uint32_t)c;
}

// q + 8 for x on the grid of step s (inv = 1 / s, rounded)
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv) {
  float q = fminf(fmaxf(rintf(x * inv), -8.f), 8.f);
  const float r = fmaf(-q, s, x), half = 0.5f * s, a = fabsf(r);
  const bool odd = ((int)q) & 1;
  if (a > half || (a == half && odd)) q += copysignf(1.f, r);
  q = fminf(fmaxf(q, -7.f), 7.f);
  return (uint32_t)((int)q + 8);
}

__device__ __forceinline__ uint32_t pack8(const uint32_t (&u)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= u[e] << ((e >> 1) * 4 + (e & 1) * 16);
  return w;
}

// Writes the positions i of one block whose s_row[i] >= 0: row s_row[i] of
// the head's k_rows / v_rows [rows, d].  xs: [16][d] floats of shared memory.
// Called by all kThreads threads; ends with a barrier.
template <typename T>
__device__ void store_block(const T* k_rows, const T* v_rows, int d, uint8_t* kb, uint8_t* vb, const int* s_row,
                            float* xs, uint32_t* s_code) {
  const int tid = threadIdx.x;
  // V: stage the rows and take each position's scale (8 threads a position)
  {
    const int i = tid >> 3, part = tid & 7;
    const int row = s_row[i];
    float amax = 0.f;
    if (row >= 0)
      for (int c = part; c < d / 8; c += 8) {
        float x[8];
        load_row8<T>(v_rows + (int64_t)row * d + c * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = no_nan(x[e]);
          amax = fmaxf(amax, fabsf(x[e]));
        }
        store_row8(xs + i * d + c * 8, x);
      }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (part == 0 && row >= 0) {
      const uint32_t code = scale_code(amax);
      s_code[i] = code;
      vb[v_scale(d, i)] = (uint8_t)code;
    }
  }
  // K: 4 lanes a group of 32 channels, 8 positions a warp
  for (int e = tid; e < 2 * d; e += kThreads) {
    const int sub = e & 3, i = (e >> 2) & 15, c = e >> 6;
    const int row = s_row[i];
    float x[8];
    float amax = 0.f;
    if (row >= 0) {
      load_row8<T>(k_rows + (int64_t)row * d + c * kGroup + sub * 8, x);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        x[t] = no_nan(x[t]);
        amax = fmaxf(amax, fabsf(x[t]));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if (row >= 0) {
      const uint32_t code = scale_code(amax);
      const float s = scale_of(code), inv = 1.f / s;
      uint32_t u[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) u[t] = code_of(x[t], s, inv);
      *reinterpret_cast<uint32_t*>(kb + k_code(c, i) + sub * 4) = pack8(u);
      if (sub == 0) kb[k_scale(d, c, i)] = (uint8_t)code;
    }
  }
  __syncthreads();
  // V: a thread per channel gathers its 16 positions
  uint32_t keep_lo = 0, keep_hi = 0;                   // nibbles of positions not written
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (s_row[i] < 0) (i < 8 ? keep_lo : keep_hi) |= 15u << (((i & 7) >> 1) * 4 + (i & 1) * 16);
  for (int ch = tid; ch < d; ch += kThreads) {
    uint2* dst = reinterpret_cast<uint2*>(vb + v_code(ch));
    uint32_t w[2] = {0u, 0u};
    if (keep_lo | keep_hi) {
      const uint2 old = __ldcg(dst);           // through L2: the line's other blocks change meanwhile
      w[0] = old.x & keep_lo;
      w[1] = old.y & keep_hi;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (s_row[i] >= 0) {
        const float s = scale_of(s_code[i]);
        w[i >> 3] |= code_of(xs[i * d + ch], s, 1.f / s) << (((i & 7) >> 1) * 4 + (i & 1) * 16);
      }
    *dst = make_uint2(w[0], w[1]);
  }
  __syncthreads();
}

// A sequence's rows for append and read: true (and its first row, count and
// first position) when they are valid and fit.  Every thread gets the same
// answer; `lead` reports.
__device__ bool seq_range(const Kv4RowsParams& p, int b, bool lead, int64_t* r0, int* n, int64_t* start) {
  const int64_t a = p.row_offsets[b], c = p.row_offsets[b + 1];
  const int64_t s = p.start[b];
  if (a < 0 || c < a || c > p.rows || c - a > p.max_rows) {
    if (lead) set_status(p.status, TV_DEV_BAD_OFFSETS);
    return false;
  }
  if (s < 0) {
    if (lead) set_status(p.status, TV_DEV_BAD_PREFIX);
    return false;
  }
  if (s + (c - a) > p.capacity) {
    if (lead) set_status(p.status, TV_DEV_CAPACITY);
    return false;
  }
  *r0 = a;
  *n = (int)(c - a);
  *start = s;
  return true;
}

// grid (blocks of the longest sequence, KV head, sequence)
template <typename T>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(const Kv4RowsParams p) {
  extern __shared__ float4 dyn[];
  __shared__ int s_row[16];
  __shared__ uint32_t s_code[16];
  dep_wait();
  dep_launch();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int64_t r0, start;
  int n;
  if (!seq_range(p, b, tid == 0 && blockIdx.x == 0 && g == 0, &r0, &n, &start)) return;
  const int64_t blk = start / kPageSize + blockIdx.x;
  if (blk * kPageSize >= start + n) return;
  uint8_t* kb = const_cast<uint8_t*>(block_at(p.k4, k_block_bytes(p.d), b, g, blk, p.Hkv, p.max_pages, p.page_table,
                                              p.num_pages));
  uint8_t* vb = const_cast<uint8_t*>(block_at(p.v4, v_block_bytes(p.d), b, g, blk, p.Hkv, p.max_pages, p.page_table,
                                              p.num_pages));
  if (!kb) {
    if (tid == 0) set_status(p.status, TV_DEV_BAD_PAGE);
    return;
  }
  if (tid < 16) {
    const int64_t i = blk * kPageSize + tid - start;
    s_row[tid] = i >= 0 && i < n ? (int)i : -1;
  }
  __syncthreads();
  const T* k = reinterpret_cast<const T*>(p.k) + ((int64_t)g * p.rows + r0) * p.d;
  const T* v = reinterpret_cast<const T*>(p.v) + ((int64_t)g * p.rows + r0) * p.d;
  store_block<T>(k, v, p.d, kb, vb, s_row, reinterpret_cast<float*>(dyn), s_code);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(const Kv4RowsParams p) {
  extern __shared__ float4 dyn[];
  float* xs = reinterpret_cast<float*>(dyn);
  dep_wait();
  dep_launch();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, d = p.d;
  int64_t r0, start;
  int n;
  if (!seq_range(p, b, tid == 0 && blockIdx.x == 0 && g == 0, &r0, &n, &start)) return;
  const int64_t blk = start / kPageSize + blockIdx.x;
  const int64_t first = blk * kPageSize - start;       // row of the block's position 0 (may be negative)
  if (first >= n) return;
  const uint8_t* kb = block_at(p.k4, k_block_bytes(d), b, g, blk, p.Hkv, p.max_pages, p.page_table, p.num_pages);
  const uint8_t* vb = block_at(p.v4, v_block_bytes(d), b, g, blk, p.Hkv, p.max_pages, p.page_table, p.num_pages);
  if (!kb) {
    if (tid == 0) set_status(p.status, TV_DEV_BAD_PAGE);
    return;
  }
  T* k = reinterpret_cast<T*>(p.k_out) + ((int64_t)g * p.rows + r0) * d;
  T* v = reinterpret_cast<T*>(p.v_out) + ((int64_t)g * p.rows + r0) * d;
  for (int ch = tid; ch < d; ch += kThreads) {
    const uint2 w = *reinterpret_cast<const uint2*>(vb + v_code(ch));
#pragma unroll
    for (int i = 0; i < 16; ++i)
      xs[i * d + ch] = (float)(nibble(i < 8 ? w.x : w.y, i & 7) - 8) * scale_of(vb[v_scale(d, i)]);
  }
  for (int e = tid; e < 2 * d; e += kThreads) {
    const int sub = e & 3, i = (e >> 2) & 15, c = e >> 6;
    const int64_t row = first + i;
    if (row < 0 || row >= n) continue;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(kb + k_code(c, i) + sub * 4);
    const float s = scale_of(kb[k_scale(d, c, i)]);
    float x[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) x[t] = (float)(nibble(w, t) - 8) * s;
    store_row8(k + row * d + c * kGroup + sub * 8, x);
  }
  __syncthreads();
  for (int e = tid; e < 2 * d; e += kThreads) {
    const int c8 = e % (d / 8), i = e / (d / 8);
    const int64_t row = first + i;
    if (row < 0 || row >= n) continue;
    const float4 lo = reinterpret_cast<const float4*>(xs + i * d + c8 * 8)[0];
    const float4 hi = reinterpret_cast<const float4*>(xs + i * d + c8 * 8)[1];
    const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    store_row8(v + row * d + c8 * 8, x);
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Walk and commit of one sequence by a cluster of CTAs (grid (C, B)): every
// CTA finds the accepted path (64 nodes at most: cheaper than passing it on),
// CTA 0 writes the outputs, and CTA c quantises the path's rows of the KV
// heads c, c + C, ...  The rule is tree_accept_commit's: node c matches when
// its draft is its parent's target argmax; the end of the path is the deepest
// node whose whole root path matches, the smallest index among equals.
template <typename T>
__global__ __launch_bounds__(kThreads) void kv4_commit_kernel(const Kv4CommitParams p) {
  extern __shared__ float4 dyn[];
  __shared__ int s_par[kMaxNodes], s_draft[kMaxNodes], s_am[kMaxNodes], s_path[kMaxNodes];
  __shared__ uint64_t s_anc[kMaxNodes];
  __shared__ uint32_t s_match[2];
  __shared__ int s_key[2], s_pid[kMaxNodes / kPageSize + 1], s_bad, s_row[16];
  __shared__ uint32_t s_code[16];
  dep_wait();
  dep_launch();
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const bool lead = blockIdx.x == 0;
  int o0 = 0, n = 0;
  const bool valid = seq_rows(p.node_offsets, b, p.R, p.max_nodes, lead && tid == 0 ? p.status : nullptr, &o0, &n);
  const int P = valid ? p.prefix_len[b] : 0;
  if (tid < n) {
    s_par[tid] = p.parents[o0 + tid];
    s_draft[tid] = p.draft[o0 + tid];
    s_am[tid] = p.argmax[o0 + tid];
  }
  if (p.page_table && valid && P >= 0 && tid < kMaxNodes / kPageSize + 1) {
    const int64_t pg = (int64_t)P / kPageSize + tid;
    s_pid[tid] = pg < p.max_pages ? p.page_table[(int64_t)b * p.max_pages + pg] : -1;
  }
  if (tid == 0) s_bad = 0;
  __syncthreads();
  uint64_t bits = 0;
  int dep = 0;
  bool match = false;
  if (tid < n) {
    int j = tid;
    bool ok = true;
    while (true) {                                     // terminates: the chain index strictly falls
      bits |= 1ull << j;
      const int q = s_par[j];
      if (j == 0) {
        ok = q == -1;
        break;
      }
      if (q < 0 || q >= j) {
        ok = false;
        break;
      }
      j = q;
      ++dep;
    }
    if (!ok) {
      bits = 1ull << tid;
      dep = 0;
      s_bad = 1;
    }
    s_anc[tid] = bits;
    match = tid == 0 || (ok && s_draft[tid] == s_am[s_par[tid]]);
  }
  if (tid < kMaxNodes) {
    const uint32_t m = __ballot_sync(0xffffffffu, match);
    if (lane == 0) s_match[tid >> 5] = m;
  }
  __syncthreads();
  const uint64_t matched = (uint64_t)s_match[0] | ((uint64_t)s_match[1] << 32);
  if (tid < kMaxNodes) {
    int key = tid < n && (bits & ~matched) == 0 ? (dep << 8) | (255 - tid) : -1;
    key = __reduce_max_sync(0xffffffffu, key);
    if (lane == 0) s_key[tid >> 5] = key;
  }
  __syncthreads();
  const int key = max(s_key[0], s_key[1]);             // >= 0 for a valid sequence: the root always matches
  const int end = 255 - (key & 255), k = key >> 8;
  if (valid && tid < n && ((s_anc[end] >> tid) & 1ull)) s_path[dep] = tid;
  __syncthreads();
  if (lead && tid < p.max_nodes) {
    const int64_t o = (int64_t)b * p.max_nodes + tid;
    p.path[o] = valid && tid <= k ? s_path[tid] : -1;
    p.tokens[o] = !valid || tid > k ? -1 : (tid < k ? s_draft[s_path[tid + 1]] : s_am[end]);
  }
  if (lead && tid == 0) {
    p.accept_len[b] = valid ? k : -1;
    if (s_bad) set_status(p.status, TV_DEV_BAD_TREE);
  }
  bool ok = valid;
  int why = 0;
  if (valid) {
    if (P < 0) {
      why = TV_DEV_BAD_PREFIX;
    } else if ((int64_t)P + k + 1 > p.capacity) {
      why = TV_DEV_CAPACITY;
    } else if (p.page_table) {
      for (int j = 0; j <= (P + k) / kPageSize - P / kPageSize; ++j)
        if (s_pid[j] < 0 || s_pid[j] >= p.num_pages) why = TV_DEV_BAD_PAGE;
    }
    if (why) {
      ok = false;
      if (lead && tid == 0) set_status(p.status, why);
    }
  }
  cluster_arrive();                                    // this CTA has read prefix_len[b]
  if (ok) {
    const int first = P / kPageSize, last = (P + k) / kPageSize;
    for (int g = blockIdx.x; g < p.Hkv; g += gridDim.x) {
      const T* kr = reinterpret_cast<const T*>(p.k_tree) + ((int64_t)g * p.R + o0) * p.d;
      const T* vr = reinterpret_cast<const T*>(p.v_tree) + ((int64_t)g * p.R + o0) * p.d;
      for (int blk = first; blk <= last; ++blk) {
        if (tid < 16) {
          const int t = blk * kPageSize + tid - P;
          s_row[tid] = t >= 0 && t <= k ? s_path[t] : -1;
        }
        __syncthreads();
        const int64_t at = p.page_table ? (int64_t)s_pid[blk - first] * p.Hkv + g
                                        : ((int64_t)b * p.Hkv + g) * p.max_pages + blk;
        store_block<T>(kr, vr, p.d, p.k4 + at * k_block_bytes(p.d), p.v4 + at * v_block_bytes(p.d), s_row,
                       reinterpret_cast<float*>(dyn), s_code);
      }
    }
  }
  cluster_wait();                                      // every CTA has read prefix_len[b]
  if (lead && tid == 0 && ok) p.prefix_len[b] = P + k + 1;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowsParams& p, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)((p.max_rows + kPageSize - 1) / kPageSize + 1), p.Hkv, p.B);
  const size_t smem = (size_t)kPageSize * p.d * 4;
  return dtype == TV_F32 ? launch_dep(kv4_append_kernel<float>, grid, dim3(kThreads), smem, s, p)
                         : launch_dep(kv4_append_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, s, p);
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)((p.max_rows + kPageSize - 1) / kPageSize + 1), p.Hkv, p.B);
  const size_t smem = (size_t)kPageSize * p.d * 4;
  return dtype == TV_F32 ? launch_dep(kv4_read_kernel<float>, grid, dim3(kThreads), smem, s, p)
                         : launch_dep(kv4_read_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, s, p);
}

cudaError_t launch_kv4_commit(const Kv4CommitParams& p, int dtype, cudaStream_t s) {
  const int C = p.Hkv < 8 ? p.Hkv : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)kPageSize * p.d * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return dtype == TV_F32 ? cudaLaunchKernelEx(&cfg, kv4_commit_kernel<float>, p)
                         : cudaLaunchKernelEx(&cfg, kv4_commit_kernel<__nv_bfloat16>, p);
}

}  // namespace tv
