// Writing and reading the 4-bit cache (include/tree_kv4.h): rows in, the
// accepted path of a verify step in, rows out.
//
// Quantisation of a group with largest magnitude A (32 channels of K, all
// channels of V at one position): the smallest scale s with 7 s >= A, then
// q = round(x / s) to even, |q| <= 7, u = q + 8, as in exact arithmetic, ties
// included.  x / s is taken as x times the reciprocal and rounded to a whole
// number by adding 1.5 x 2^23 (no conversion instruction: those run at a
// quarter of the rate).  An fp32 value's result is then corrected by the exact
// residual x - q s (it has no more bits than x); a bf16 value needs none
// (steps_of).  The sum's low bits are q, so eight of them pack by
// multiply-adds.
//
// One CTA handles the 16-position block of one KV head, K and V, and issues
// all its loads before the first use.  K is quantised where it is loaded: four
// lanes hold a position's 32-channel group and share its maximum.  V's codes
// run along the positions, so its 16 rows are staged in shared memory once and
// read back by channel; a block that is written in part keeps the other
// positions' nibbles.  Reading expands pairs as the attention does (mask and
// one bf16 fused multiply-add, exact) and turns V back through shared memory.
// Nothing is read twice.  Four prompts of up to 32768 rows (8 KV heads of 128,
// bf16): writing 107 us, 517 MB, 4.8 TB/s, bound by issue slots (81%: about
// eight instructions a value with addresses and scales); reading back 91 us,
// 5.7 TB/s, bound by memory.
#include "tv_kv4.cuh"
#include "tv_kv4_store.cuh"

namespace tv {
namespace {

using namespace kv4;

constexpr int kThreads = 128;

// 8 values of a row in global memory, raw (through L2: rows are read once)
template <typename T>
struct Row8;

template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = __ldcg(reinterpret_cast<const float4*>(src));
    b = __ldcg(reinterpret_cast<const float4*>(src) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  // largest magnitude as bits: above 0x7f800000 where a value is NaN
  __device__ __forceinline__ uint32_t top() const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void tame(float most);
  __device__ __forceinline__ void store(float* dst) const {        // to shared memory
    reinterpret_cast<float4*>(dst)[0] = a;
    reinterpret_cast<float4*>(dst)[1] = b;
  }
};

template <>
struct Row8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* src) { u = __ldcg(reinterpret_cast<const uint4*>(src)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[2 * t] = __uint_as_float(w[t] << 16);
      x[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ void tame(float most);
  __device__ __forceinline__ void store(__nv_bfloat16* dst) const { *reinterpret_cast<uint4*>(dst) = u; }
};

// The rare groups: a value that is not a number counts as 0, magnitudes end
// at `most` (7 steps of the largest scale, a bf16 number too).
__device__ __forceinline__ float tame1(float x, float most) { return x != x ? 0.f : fminf(fmaxf(x, -most), most); }
__device__ __forceinline__ void Row8<float>::tame(float most) {
  a = make_float4(tame1(a.x, most), tame1(a.y, most), tame1(a.z, most), tame1(a.w, most));
  b = make_float4(tame1(b.x, most), tame1(b.y, most), tame1(b.z, most), tame1(b.w, most));
}
__device__ __forceinline__ void Row8<__nv_bfloat16>::tame(float most) {
  uint32_t* w = &u.x;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t lo = __float_as_uint(tame1(__uint_as_float(w[t] << 16), most));
    const uint32_t hi = __float_as_uint(tame1(__uint_as_float(w[t] & 0xffff0000u), most));
    w[t] = (lo >> 16) | (hi & 0xffff0000u);
  }
}
constexpr float kMost = 7.f * 65536.f * 1.875f;  // 7 steps of the largest scale

// two adjacent values of a staged row
__device__ __forceinline__ void two(const float* p, float& x, float& y) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x = v.x;
  y = v.y;
}
__device__ __forceinline__ void two(const __nv_bfloat16* p, float& x, float& y) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  x = __uint_as_float(w << 16);
  y = __uint_as_float(w & 0xffff0000u);
}

// smallest code whose 7 steps reach amax <= kMost: the code below amax / 7
// (taken a little low, so never above the answer's predecessor), and one more
// for each of the next two that still falls short (7 s is exact)
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const int bits = __float_as_int(amax * (0.99999f / 7.f));
  const uint32_t c = (uint32_t)max((bits >> 20) - (112 << 3), 0);
  const float s = scale_of(c), next = scale_of(c + 1);
  return c + (7.f * s < amax ? 1u : 0u) + (7.f * next < amax ? 1u : 0u);
}

// 1 / s within 2^-22 (steps_of allows for more)
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

constexpr float kMagic = 12582912.f;             // 1.5 x 2^23: x + kMagic is x rounded to a whole number
constexpr uint32_t kMagicBits = 0x4B400000u;

// bits kMagicBits + q of x on the grid of step s (inv = 1 / s within 2^-22); |x| <= 7 s
template <typename T>
__device__ __forceinline__ uint32_t steps_of(float x, float s, float inv);
template <>
__device__ __forceinline__ uint32_t steps_of<float>(float x, float s, float inv) {
  float t = fmaf(x, inv, kMagic);
  const float r = fmaf(kMagic - t, s, x);
  // too far, or half way with an odd q: one step on (the bound is s / 2, and for an odd q the float below it)
  const float bound = __uint_as_float(__float_as_uint(0.5f * s) - (__float_as_uint(t) & 1u));
  if (fabsf(r) > bound) t += copysignf(1.f, r);
  return __float_as_uint(t);
}
// x is a bf16 number: x / s = X 2^k / (8 + m) with X < 256.  Where that is near
// a half (2 q + 1) / 2 it is the half, or at least 2^(k + 1) / (2 (8 + m)) away
// with k >= -6: more than 2^-10.  So rounding x inv (off by 7 x 2^-22 at most)
// to the grid of 2^-13 first finds each half exactly and moves nothing across
// one; the second sum then rounds to whole numbers, halves to even.
template <>
__device__ __forceinline__ uint32_t steps_of<__nv_bfloat16>(float x, float, float inv) {
  constexpr float kFine = 1536.f;                // 1.5 x 2^10: the sum's last bit is 2^-13
  return __float_as_uint(fmaf(x, inv, kFine) + (kMagic - kFine));
}

__host__ __device__ constexpr int value_bit(int e) { return (e >> 1) * 4 + (e & 1) * 16; }

// sum over e of (kMagicBits + 8's complement) << bit(e): what pack leaves on top of the codes q + 8
__host__ __device__ constexpr uint32_t pack_excess() {
  uint32_t c = 0;
  for (int e = 0; e < 8; ++e) c += (kMagicBits - 8u) << value_bit(e);
  return c;
}

// Writes the positions i of one block whose s_row[i] >= 0 (one at least: row 0
// is read in place of the others): row s_row[i] of the head's k_rows / v_rows
// [rows, D].  xs: [16][D] of shared memory.
// Called by all kThreads threads; ends with a barrier.
template <typename T, int D>
__device__ __forceinline__ void store_block(const T* k_rows, const T* v_rows, uint8_t* kb, uint8_t* vb, const int* s_row,
                                            T* xs, float2* s_step) {
  constexpr int IT = D / 64;                     // 8-value pieces per thread, of K and of V
  const int tid = threadIdx.x;
  Row8<T> kx[IT], vx[IT];
  // (a position not written loads row 0 and drops what comes of it)
  const int vi = tid >> 3, vrow = s_row[vi];
#pragma unroll
  for (int q = 0; q < IT; ++q) vx[q].load(v_rows + (int64_t)max(vrow, 0) * D + ((tid & 7) + 8 * q) * 8);
  const int ki = (tid >> 2) & 15, krow = s_row[ki];   // the same position in each piece
#pragma unroll
  for (int q = 0; q < IT; ++q) {
    const int c = (tid >> 6) + 2 * q;
    kx[q].load(k_rows + (int64_t)max(krow, 0) * D + c * kGroup + (tid & 3) * 8);
  }
  const uint32_t gone = __ballot_sync(0xffffffffu, s_row[tid & 15] < 0) & 0xffffu;   // positions not written
  // V: stage the rows and take each position's scale (8 threads a position)
  {
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < IT; ++q) top = max(top, vx[q].top());
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (top > __float_as_uint(kMost)) {                // NaN, infinity or beyond the largest scale
      top = 0;
#pragma unroll
      for (int q = 0; q < IT; ++q) {
        vx[q].tame(kMost);
        top = max(top, vx[q].top());
      }
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) top = max(top, __shfl_xor_sync(0xffu << (tid & 24), top, off));
    }
#pragma unroll
    for (int q = 0; q < IT; ++q) vx[q].store(xs + vi * D + ((tid & 7) + 8 * q) * 8);
    if ((tid & 7) == 0) {
      const uint32_t code = scale_code(__uint_as_float(top));
      const float s = scale_of(code);
      s_step[vi] = make_float2(s, reciprocal(s));
      if (vrow >= 0) vb[v_scale(D, vi)] = (uint8_t)code;
    }
  }
  // K: 4 lanes a group of 32 channels, 8 positions a warp
#pragma unroll
  for (int q = 0; q < IT; ++q) {
    const int sub = tid & 3, c = (tid >> 6) + 2 * q;
    uint32_t top = kx[q].top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (top > __float_as_uint(kMost)) {
      kx[q].tame(kMost);
      top = kx[q].top();
      top = max(top, __shfl_xor_sync(0xfu << (tid & 28), top, 1));
      top = max(top, __shfl_xor_sync(0xfu << (tid & 28), top, 2));
    }
    if (krow >= 0) {
      const uint32_t code = scale_code(__uint_as_float(top));
      const float s = scale_of(code), inv = reciprocal(s);
      float x[8];
      kx[q].get(x);
      uint32_t w = 0;
#pragma unroll
      for (int t = 0; t < 8; ++t) w += steps_of<T>(x[t], s, inv) << value_bit(t);
      *reinterpret_cast<uint32_t*>(kb + k_code(c, ki) + sub * 4) = w - pack_excess();
      if (sub == 0) kb[k_scale(D, c, ki)] = (uint8_t)code;
    }
  }
  __syncthreads();
  // V: a thread gathers 8 positions (half h of the block) of two channels
  const int h = tid >> 6;
  uint32_t keep = 0;                                   // nibbles of positions not written
  if (gone) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((gone >> (8 * h + i)) & 1u) keep |= 15u << value_bit(i);
  }
#pragma unroll 1
  for (int ch = 2 * (tid & 63); ch < D; ch += kThreads) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 st = s_step[8 * h + i];
      float x, y;
      two(xs + (8 * h + i) * D + ch, x, y);
      w[0] += steps_of<T>(x, st.x, st.y) << value_bit(i);
      w[1] += steps_of<T>(y, st.x, st.y) << value_bit(i);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(vb + v_code(ch + e)) + h;
      w[e] -= pack_excess();
      if (keep) w[e] = (w[e] & ~keep) | (__ldcg(dst) & keep);      // through L2: the line's other blocks change meanwhile
      *dst = w[e];
    }
  }
  __syncthreads();
}

// A sequence's rows for append and read: true (and its first row, count and
// first position) when there are any, they are valid and fit.  A sequence
// without rows touches nothing: it has no row 0 that store_block could load,
// and its start may name a block that another sequence writes, or no page.
// Every thread gets the same answer; `lead` reports.
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
  return c > a;
}

// grid (blocks of the longest sequence, KV head, sequence)
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_append_kernel(const Kv4RowsParams p) {
  __shared__ __align__(16) T xs[16 * D];
  __shared__ int s_row[16];
  __shared__ float2 s_step[16];
  dep_wait();
  dep_launch();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int64_t r0, start;
  int n;
  if (!seq_range(p, b, tid == 0 && blockIdx.x == 0 && g == 0, &r0, &n, &start)) return;
  const int64_t blk = start / kPageSize + blockIdx.x;
  if (blk * kPageSize >= start + n) return;
  uint8_t* kb = const_cast<uint8_t*>(block_at(p.k4, k_block_bytes(D), b, g, blk, p.Hkv, p.max_pages, p.page_table,
                                              p.num_pages));
  uint8_t* vb = const_cast<uint8_t*>(block_at(p.v4, v_block_bytes(D), b, g, blk, p.Hkv, p.max_pages, p.page_table,
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
  const T* k = reinterpret_cast<const T*>(p.k) + ((int64_t)g * p.rows + r0) * D;
  const T* v = reinterpret_cast<const T*>(p.v) + ((int64_t)g * p.rows + r0) * D;
  store_block<T, D>(k, v, kb, vb, s_row, xs, s_step);
}

// pair j of a word times the bf16 pair of scales s2, exact
__device__ __forceinline__ uint32_t pair_value(uint32_t w, int j, uint32_t s2) {
  return fma_bf16x2(((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u, s2, fma_bf16x2(s2, kMinus136, kMinusZero));
}
__device__ __forceinline__ uint32_t scale_bits(uint32_t code) { return (code << 4) + 0x3800u; }   // as bf16

// 8 bf16 values to a row
__device__ __forceinline__ void put8(__nv_bfloat16* dst, const uint4& u) { *reinterpret_cast<uint4*>(dst) = u; }
__device__ __forceinline__ void put8(float* dst, const uint4& u) {
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(u.x << 16, u.x & 0xffff0000u, u.y << 16, u.y & 0xffff0000u);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(u.z << 16, u.z & 0xffff0000u, u.w << 16, u.w & 0xffff0000u);
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(const Kv4RowsParams p) {
  constexpr int IT = D / 64, PITCH = D + 8;      // (the pad keeps 16-byte rows and spreads the banks)
  __shared__ __align__(16) uint16_t xs[16 * PITCH];
  dep_wait();
  dep_launch();
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int64_t r0, start;
  int n;
  if (!seq_range(p, b, tid == 0 && blockIdx.x == 0 && g == 0, &r0, &n, &start)) return;
  const int64_t blk = start / kPageSize + blockIdx.x;
  const int64_t first = blk * kPageSize - start;       // row of the block's position 0 (may be negative)
  if (first >= n) return;
  const uint8_t* kb = block_at(p.k4, k_block_bytes(D), b, g, blk, p.Hkv, p.max_pages, p.page_table, p.num_pages);
  const uint8_t* vb = block_at(p.v4, v_block_bytes(D), b, g, blk, p.Hkv, p.max_pages, p.page_table, p.num_pages);
  if (!kb) {
    if (tid == 0) set_status(p.status, TV_DEV_BAD_PAGE);
    return;
  }
  T* k = reinterpret_cast<T*>(p.k_out) + ((int64_t)g * p.rows + r0) * D;
  T* v = reinterpret_cast<T*>(p.v_out) + ((int64_t)g * p.rows + r0) * D;
  // every load first
  constexpr int CT = D / kThreads;               // V channels per thread
  uint2 vw[CT];
  uint32_t kw[IT], kc[IT];
  const uint4 vsc = __ldcg(reinterpret_cast<const uint4*>(vb + v_scale(D, 0)));
#pragma unroll
  for (int q = 0; q < CT; ++q) vw[q] = __ldcg(reinterpret_cast<const uint2*>(vb + v_code(tid + q * kThreads)));
#pragma unroll
  for (int q = 0; q < IT; ++q) {
    const int e = tid + q * kThreads, sub = e & 3, i = (e >> 2) & 15, c = e >> 6;
    kw[q] = __ldcg(reinterpret_cast<const uint32_t*>(kb + k_code(c, i)) + sub);
    kc[q] = __ldcg(kb + k_scale(D, c, i));
  }
#pragma unroll
  for (int q = 0; q < CT; ++q) {
    const uint32_t sc[4] = {vsc.x, vsc.y, vsc.z, vsc.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {                      // positions 2 j, 2 j + 1
      const uint32_t two = sc[j >> 1] >> (16 * (j & 1));
      const uint32_t s2 = scale_bits(two & 255u) | (scale_bits((two >> 8) & 255u) << 16);
      const uint32_t x = pair_value(j < 4 ? vw[q].x : vw[q].y, j & 3, s2);
      xs[(2 * j) * PITCH + tid + q * kThreads] = (uint16_t)x;
      xs[(2 * j + 1) * PITCH + tid + q * kThreads] = (uint16_t)(x >> 16);
    }
  }
#pragma unroll
  for (int q = 0; q < IT; ++q) {
    const int e = tid + q * kThreads, sub = e & 3, i = (e >> 2) & 15, c = e >> 6;
    const int64_t row = first + i;
    if (row < 0 || row >= n) continue;
    const uint32_t s2 = scale_bits(kc[q]) * 0x00010001u;
    put8(k + row * D + c * kGroup + sub * 8, make_uint4(pair_value(kw[q], 0, s2), pair_value(kw[q], 1, s2),
                                                        pair_value(kw[q], 2, s2), pair_value(kw[q], 3, s2)));
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < IT; ++q) {
    const int e = tid + q * kThreads, c8 = e % (D / 8), i = e / (D / 8);
    const int64_t row = first + i;
    if (row < 0 || row >= n) continue;
    put8(v + row * D + c8 * 8, *reinterpret_cast<const uint4*>(xs + i * PITCH + c8 * 8));
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
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void kv4_commit_kernel(const Kv4CommitParams p) {
  __shared__ __align__(16) T xs[16 * D];
  __shared__ int s_par[kMaxNodes], s_draft[kMaxNodes], s_am[kMaxNodes], s_path[kMaxNodes];
  __shared__ uint64_t s_anc[kMaxNodes];
  __shared__ uint32_t s_match[2];
  __shared__ int s_key[2], s_pid[kMaxNodes / kPageSize + 1], s_bad, s_row[16];
  __shared__ float2 s_step[16];
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
      const T* kr = reinterpret_cast<const T*>(p.k_tree) + ((int64_t)g * p.R + o0) * D;
      const T* vr = reinterpret_cast<const T*>(p.v_tree) + ((int64_t)g * p.R + o0) * D;
      for (int blk = first; blk <= last; ++blk) {
        if (tid < 16) {
          const int t = blk * kPageSize + tid - P;
          s_row[tid] = t >= 0 && t <= k ? s_path[t] : -1;
        }
        __syncthreads();
        const int64_t at = p.page_table ? (int64_t)s_pid[blk - first] * p.Hkv + g
                                        : ((int64_t)b * p.Hkv + g) * p.max_pages + blk;
        store_block<T, D>(kr, vr, p.k4 + at * k_block_bytes(D), p.v4 + at * v_block_bytes(D), s_row, xs, s_step);
      }
    }
  }
  cluster_wait();                                      // every CTA has read prefix_len[b]
  if (lead && tid == 0 && ok) p.prefix_len[b] = P + k + 1;
}

}  // namespace

// kernel<T, D> for a dtype and head_dim
#define TV_KV4_PICK(kernel, dtype, d)                                                                     \
  ((dtype) == TV_F32 ? ((d) == 128 ? kernel<float, 128> : ((d) == 256 ? kernel<float, 256> : kernel<float, 512>)) \
                     : ((d) == 128 ? kernel<__nv_bfloat16, 128>                                           \
                                   : ((d) == 256 ? kernel<__nv_bfloat16, 256> : kernel<__nv_bfloat16, 512>)))

cudaError_t launch_kv4_append(const Kv4RowsParams& p, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)((p.max_rows + kPageSize - 1) / kPageSize + 1), p.Hkv, p.B);
  return launch_dep(TV_KV4_PICK(kv4_append_kernel, dtype, p.d), grid, dim3(kThreads), 0, s, p);
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)((p.max_rows + kPageSize - 1) / kPageSize + 1), p.Hkv, p.B);
  return launch_dep(TV_KV4_PICK(kv4_read_kernel, dtype, p.d), grid, dim3(kThreads), 0, s, p);
}

cudaError_t launch_kv4_commit(const Kv4CommitParams& p, int dtype, cudaStream_t s) {
  const int C = p.Hkv < 8 ? p.Hkv : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, p.B);
  cfg.blockDim = dim3(kThreads);
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
  return cudaLaunchKernelEx(&cfg, TV_KV4_PICK(kv4_commit_kernel, dtype, p.d), p);
}

}  // namespace tv
