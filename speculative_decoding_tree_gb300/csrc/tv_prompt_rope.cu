// Prompt RoPE with the writes of keys and values (include/tree_prompt.h).
//
// A CTA takes a few rows.  Their sequences, positions and cache places are
// found first; then each row's d / 2 angles, as fractions of a turn in 64-bit
// fixed point (position * theta^(-2j/d) / 2 pi modulo 1 is one integer
// multiplication; float64 arithmetic is slow on this part), give sines and
// cosines in shared memory that every head of the row uses.  The rest is
// copies of 16 bytes: a thread turns the pairs j .. j + 7 (bf16; 3, fp32) of a
// head, whose halves are d / 2 apart.  Bound by the bytes: q read and written,
// k and v read once and written to the rows and to the cache.
#include <cmath>
#include <cstring>

#include "tv_host.cuh"
#include "tv_prompt.cuh"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 4;                         // rows of a CTA

struct PRopeParams {
  const void* q_in;
  const void* k_in;
  const void* v_in;
  const int32_t* prefix_len;
  const int32_t* row_offsets;
  void* q_out;
  void* k_rows;
  void* v_rows;
  void* k_cache;
  void* v_cache;
  const int32_t* page_table;
  int32_t* new_prefix_len;
  int32_t* status;
  int B, Hq, Hkv, d, rows_per_cta;
  int64_t rows, max_rows, capacity, num_pages, max_prefix;
  uint64_t turns[256];       // theta^(-2j/d) / 2 pi as a 64-bit fraction
};

// A sequence's prefix length as the rotation uses it; false when the sequence
// is skipped (with a cache: out of range, or its rows do not fit).
__device__ bool rope_prefix(const PRopeParams& p, int b, int64_t n, int64_t* P) {
  const int64_t raw = p.prefix_len[b];
  *P = clamp_prefix(raw, p.max_prefix, p.capacity);
  if (*P != raw) set_status(p.status, TV_DEV_BAD_PREFIX);
  if (!p.k_cache) return true;
  if (*P != raw) return false;
  if (*P + n > p.capacity) {
    set_status(p.status, TV_DEV_CAPACITY);
    return false;
  }
  return true;
}

template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;            // elements of 16 bytes
  float x[N];
  __device__ __forceinline__ void from(const uint4& w) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        x[2 * i] = __uint_as_float(a[i] << 16);
        x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(a[i]);
      }
    }
  }
  __device__ __forceinline__ uint4 to() const {
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : __float_as_uint(x[i]);
    return make_uint4(a[0], a[1], a[2], a[3]);
  }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) prompt_rope_kernel(const __grid_constant__ PRopeParams p) {
  constexpr int N = Vec<BF16>::N, ES = BF16 ? 2 : 4;
  __shared__ float2 s_cs[kMaxRows * 256];
  __shared__ int64_t s_pos[kMaxRows], s_cache[kMaxRows];   // position (-1: skip), first cache row (-1: none)
  const int tid = threadIdx.x;
  dep_wait();
  dep_launch();
  if (blockIdx.x == gridDim.x - 1) {
    // the last CTA: every sequence's new length
    for (int b = tid; b < p.B; b += kThreads) {
      int64_t o0, n, P;
      const bool ok = prompt_rows(p.row_offsets, b, p.rows, p.max_rows, p.status, &o0, &n) && n > 0 &&
                      rope_prefix(p, b, n, &P);
      const bool fits = ok && P + n <= INT32_MAX;   // (without a cache the rows may go further than a length can)
      if (p.new_prefix_len) {
        if (ok && !fits) set_status(p.status, TV_DEV_CAPACITY);
        p.new_prefix_len[b] = fits ? (int)(P + n) : p.prefix_len[b];
      }
    }
    return;
  }
  const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_cta;
  const int nr = (int)min((int64_t)p.rows_per_cta, p.rows - r0);
  if (tid < nr) {
    const int64_t r = r0 + tid;
    int lo = 0, hi = p.B;                           // the last sequence that starts at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.row_offsets[mid] <= r) lo = mid;
      else hi = mid;
    }
    int64_t o0, n, P, pos = -1, at = -1;
    if (prompt_rows(p.row_offsets, lo, p.rows, p.max_rows, p.status, &o0, &n) && r >= o0 && r < o0 + n &&
        rope_prefix(p, lo, n, &P)) {
      pos = P + (r - o0);
      if (p.k_cache && p.page_table) {
        const int pid = p.page_table[(int64_t)lo * (p.capacity / kPageSize) + pos / kPageSize];
        if (pid >= 0 && pid < p.num_pages) at = (int64_t)pid * p.Hkv * kPageSize + pos % kPageSize;
        else set_status(p.status, TV_DEV_BAD_PAGE);
      } else if (p.k_cache) {
        at = (int64_t)lo * p.Hkv * p.capacity + pos;
      }
    }
    s_pos[tid] = pos;
    s_cache[tid] = at;
  }
  __syncthreads();
  const int half = p.d / 2;
  for (int e = tid; e < nr * half; e += kThreads) {
    const int r = e / half, j = e - r * half;
    if (s_pos[r] < 0) continue;
    const uint64_t t = (uint64_t)s_pos[r] * p.turns[j];
    // the turn as a signed fraction in [-1/2, 1/2): its top 32 bits, in half turns
    const float x = (float)(int32_t)(t >> 32) * (1.f / 2147483648.f);
    float sn, cs;
    sincospif(x, &sn, &cs);
    s_cs[r * half + j] = make_float2(cs, sn);
  }
  __syncthreads();
  const int64_t head_rows = p.page_table ? kPageSize : p.capacity;   // cache rows from one KV head to the next
  const int hv = half / N, heads = p.Hq + p.Hkv;
  // tasks: (row, head, vector of the half), queries then keys
  for (int e = tid; e < nr * heads * hv; e += kThreads) {
    const int r = e / (heads * hv), h = e / hv % heads, v = e % hv;
    if (s_pos[r] < 0) continue;
    const bool isq = h < p.Hq;
    const int64_t in = isq ? ((r0 + r) * p.Hq + h) * p.d : ((r0 + r) * p.Hkv + h - p.Hq) * p.d;
    const char* src = reinterpret_cast<const char*>(isq ? p.q_in : p.k_in) + (in + v * N) * ES;
    Vec<BF16> a, b;
    a.from(*reinterpret_cast<const uint4*>(src));
    b.from(*reinterpret_cast<const uint4*>(src + half * ES));
    Vec<BF16> lo, hi;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 c = s_cs[r * half + v * N + i];
      lo.x[i] = a.x[i] * c.x - b.x[i] * c.y;
      hi.x[i] = b.x[i] * c.x + a.x[i] * c.y;
    }
    const uint4 wl = lo.to(), wh = hi.to();
    auto store = [&](void* base, int64_t elem) {
      char* dst = reinterpret_cast<char*>(base) + (elem + v * N) * ES;
      *reinterpret_cast<uint4*>(dst) = wl;
      *reinterpret_cast<uint4*>(dst + half * ES) = wh;
    };
    if (isq) {
      store(p.q_out, in);
    } else {
      const int g = h - p.Hq;
      if (p.k_rows) store(p.k_rows, ((int64_t)g * p.rows + r0 + r) * p.d);
      if (s_cache[r] >= 0) store(p.k_cache, (s_cache[r] + g * head_rows) * p.d);
    }
  }
  const int dv = p.d / N;
  for (int e = tid; e < nr * p.Hkv * dv; e += kThreads) {
    const int r = e / (p.Hkv * dv), g = e / dv % p.Hkv, v = e % dv;
    if (s_pos[r] < 0) continue;
    const uint4 w = reinterpret_cast<const uint4*>(p.v_in)[((r0 + r) * p.Hkv + g) * dv + v];
    if (p.v_rows) reinterpret_cast<uint4*>(p.v_rows)[((int64_t)g * p.rows + r0 + r) * dv + v] = w;
    if (s_cache[r] >= 0) reinterpret_cast<uint4*>(p.v_cache)[(s_cache[r] + g * head_rows) * dv + v] = w;
  }
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_prompt_rope_store(const tv_desc* desc, int64_t rows, int64_t max_rows, double theta, const void* d_q_in,
                         const void* d_k_in, const void* d_v_in, const int32_t* d_prefix_len,
                         const int32_t* d_row_offsets, void* d_q_out, void* d_k_rows, void* d_v_rows,
                         void* d_k_cache, void* d_v_cache, const int32_t* d_page_table, int32_t* d_new_prefix_len,
                         int32_t* d_status, void* stream) {
  int64_t t;
  const int rc = validate_prompt(desc, rows, max_rows);
  if (rc) return rc;
  if (!(theta > 1.0) || !std::isfinite(theta)) return TV_ERR_SHAPE;
  if (!mul_ok(rows, (int64_t)desc->num_q_heads * desc->head_dim, &t)) return TV_ERR_OVERFLOW;
  if (rows == 0 || max_rows == 0) return TV_OK;
  if (!d_q_in || !d_k_in || !d_v_in || !d_prefix_len || !d_row_offsets || !d_q_out || !d_status ||
      !d_k_rows != !d_v_rows || !d_k_cache != !d_v_cache ||
      (d_k_cache && desc->page_size == kPageSize && !d_page_table))
    return TV_ERR_NULL;
  const void* all[] = {d_q_in,   d_k_in,    d_v_in,    d_prefix_len, d_row_offsets,    d_q_out, d_k_rows,
                       d_v_rows, d_k_cache, d_v_cache, d_page_table, d_new_prefix_len, d_status};
  for (const void* x : all)
    if (!aligned16(x)) return TV_ERR_ALIGN;
  if (d_new_prefix_len == d_prefix_len) return TV_ERR_SHAPE;   // other rows still read the old lengths
  PRopeParams p = {};
  p.q_in = d_q_in; p.k_in = d_k_in; p.v_in = d_v_in;
  p.prefix_len = d_prefix_len; p.row_offsets = d_row_offsets;
  p.q_out = d_q_out; p.k_rows = d_k_rows; p.v_rows = d_v_rows; p.k_cache = d_k_cache; p.v_cache = d_v_cache;
  p.page_table = desc->page_size ? d_page_table : nullptr;
  p.new_prefix_len = d_new_prefix_len; p.status = d_status;
  p.B = desc->batch; p.Hq = desc->num_q_heads; p.Hkv = desc->num_kv_heads; p.d = desc->head_dim;
  p.rows = rows;
  p.max_rows = max_rows < rows ? max_rows : rows;
  p.capacity = desc->capacity; p.num_pages = desc->num_pages; p.max_prefix = desc->max_prefix;
  // the host's last table: its powers take longer than the launch of a short call
  static thread_local struct {
    double theta;
    int d;
    uint64_t turns[256];
  } last = {0.0, 0, {}};
  if (last.theta != theta || last.d != p.d) {
    for (int j = 0; j < p.d / 2; ++j)
      last.turns[j] = (uint64_t)(std::pow(theta, -2.0 * j / p.d) * 0.15915494309189535 * 18446744073709551616.0);
    last.theta = theta;
    last.d = p.d;
  }
  std::memcpy(p.turns, last.turns, sizeof(uint64_t) * (p.d / 2));
  // one row a CTA while that leaves SMs idle, then four
  p.rows_per_cta = rows >= (int64_t)8 * num_sms() ? kMaxRows : 1;
  const unsigned grid = (unsigned)((rows + p.rows_per_cta - 1) / p.rows_per_cta + 1);
  const cudaStream_t s = as_stream(stream);
  const cudaError_t e = desc->dtype == TV_BF16
                            ? launch_dep(prompt_rope_kernel<true>, dim3(grid), dim3(kThreads), 0, s, p)
                            : launch_dep(prompt_rope_kernel<false>, dim3(grid), dim3(kThreads), 0, s, p);
  return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // extern "C"
