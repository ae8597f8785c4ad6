// The control of tree logits (include/tree_logits.h): penalties, biases and
// grammar masks on every tree row, and the token counts they read.
//
// process: a CTA takes 2048 tokens of one sequence and several of its tree
// rows.  What the rows share is read once: a thread keeps its 8 tokens'
// counts and biases in registers (the sparse bias list goes through a table of
// entry numbers in shared memory, where the larger number wins).  What differs
// from row to row, the drafts on the path, is a table of bytes in shared
// memory; three of them in turn, so that one barrier a row separates clearing,
// filling and reading.  The next row's logits are loaded before this row's are
// stored.  Tokens that nothing touches are copied as they are.  Bound by the
// bytes: logits read and written.
#include <type_traits>

#include "tree_logits.h"
#include "tv_host.cuh"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                             // tokens a thread
constexpr int kChunk = kThreads * kPer;

struct LogitsParams {
  const void* in;
  void* out;
  const uint16_t* counts;
  const float* penalties;
  const int32_t* bias_offsets;
  const int32_t* bias_tokens;
  const float* bias_values;
  const uint32_t* mask;
  const int32_t* draft;
  const int32_t* node_offsets;
  const uint64_t* anc;
  int32_t* status;
  int B, V, R, max_nodes, biases, chunks, groups, group_rows;
};

// One token of one row: x after the penalties and the bias.
__device__ __forceinline__ float steer(float x, unsigned word, unsigned path, float rho, float phi, float pi,
                                       float bias) {
  const unsigned n = (word & 0x7fffu) + path;
  if ((word & 0x8000u) || n) x = x > 0.f ? x / rho : x * rho;
  if (n) x = x - phi * (float)n - pi;
  return x + bias;
}

// VEC: rows start on 16 bytes and a thread's 8 tokens are neighbours; else a
// warp's 256 tokens are read 32 at a time.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
  using T = typename std::conditional<BF16, uint16_t, uint32_t>::type;
  constexpr T kMinusInf = (T)(BF16 ? 0xff80u : 0xff800000u);
  __shared__ __align__(16) int s_entry[kChunk];
  __shared__ __align__(16) uint8_t s_path[3][kChunk];
  __shared__ int s_draft[64];
  __shared__ uint64_t s_anc[64];
  const int tid = threadIdx.x, lane = tid & 31;
  dep_wait();
  dep_launch();
  const int c = blockIdx.x % p.chunks;
  const int grp = blockIdx.x / p.chunks % p.groups;
  const int b = blockIdx.x / p.chunks / p.groups;
  int o0, n;
  if (!seq_rows(p.node_offsets, b, p.R, p.max_nodes, p.status, &o0, &n)) return;
  const int r0 = grp * p.group_rows, r1 = min(n, r0 + p.group_rows);
  if (r0 >= r1) return;
  const int base = c * kChunk;                      // the chunk's first token (V <= 2^30)
  const int first = base + (VEC ? tid * kPer : (tid >> 5) * 256 + lane);
  constexpr int kStep = VEC ? 1 : 32;               // from one of the thread's tokens to the next
  const int words = (p.V + 31) / 32;

  __align__(16) T x[kPer], nx[kPer];
  unsigned bits = 0xffu, nbits = 0xffu;             // the mask's bits of the thread's tokens
  auto load = [&](int r, T* dst, unsigned* m) {
    const int64_t row = (int64_t)(o0 + r) * p.V;
    const T* src = reinterpret_cast<const T*>(p.in) + row + first;
    if (VEC) {
      if (first < p.V) {
        if (BF16) {
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        } else {
          reinterpret_cast<uint4*>(dst)[0] = reinterpret_cast<const uint4*>(src)[0];
          reinterpret_cast<uint4*>(dst)[BF16 ? 0 : 1] = reinterpret_cast<const uint4*>(src)[BF16 ? 0 : 1];
        }
        if (p.mask) *m = reinterpret_cast<const uint8_t*>(p.mask + (int64_t)(o0 + r) * words)[first / 8];
      }
    } else {
      unsigned got = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = first + e * 32;
        dst[e] = v < p.V ? src[e * 32] : (T)0;
        if (p.mask && v < p.V) got |= (p.mask[(int64_t)(o0 + r) * words + v / 32] >> (v & 31) & 1u) << e;
      }
      if (p.mask) *m = got;
    }
  };
  load(r0, x, &bits);

  // what the sequence's rows share
  unsigned cnt[kPer];
  float bias[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    cnt[e] = 0;
    bias[e] = 0.f;
  }
  float rho = 1.f, phi = 0.f, pi = 0.f;
  const bool counted = p.counts != nullptr, paths = counted && p.draft != nullptr;
  if (counted) {
    rho = p.penalties[b * 3];
    phi = p.penalties[b * 3 + 1];
    pi = p.penalties[b * 3 + 2];
    const uint16_t* row = p.counts + (int64_t)b * ((p.V + 7) / 8 * 8) + first;
    if (VEC) {
      if (first < p.V) {
        const uint4 w = *reinterpret_cast<const uint4*>(row);
        const unsigned a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < kPer; ++e) cnt[e] = a[e / 2] >> (16 * (e & 1)) & 0xffffu;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (first + e * 32 < p.V) cnt[e] = row[e * 32];
    }
  }
  int nb = 0, b0 = 0;
  if (p.bias_offsets) {
    b0 = p.bias_offsets[b];
    const int64_t more = (int64_t)p.bias_offsets[b + 1] - b0;
    if (b0 < 0 || more < 0 || b0 + more > p.biases) {
      if (tid == 0) set_status(p.status, TV_DEV_BAD_OFFSETS);
    } else {
      nb = (int)more;
    }
  }
  if (nb > 0) {
    for (int e = tid; e < kChunk / 4; e += kThreads) reinterpret_cast<int4*>(s_entry)[e] = make_int4(-1, -1, -1, -1);
  }
  if (paths) {
    for (int e = tid; e < 3 * kChunk / 16; e += kThreads)
      reinterpret_cast<uint4*>(&s_path[0][0])[e] = make_uint4(0, 0, 0, 0);
    if (tid < n) {
      s_draft[tid] = p.draft[o0 + tid];
      s_anc[tid] = p.anc[o0 + tid];
    }
  }
  __syncthreads();
  for (int e = tid; e < nb; e += kThreads) {
    const int64_t t = (int64_t)p.bias_tokens[b0 + e];
    if (t < 0 || t >= p.V) {
      if (c == 0) set_status(p.status, TV_DEV_BAD_TOKEN);
    } else if (t >= base && t < base + kChunk) {
      atomicMax(&s_entry[t - base], e);
    }
  }
  // bytes of row r's path in table t, added or taken away
  auto put_path = [&](int r, int t, bool add) {
    if (tid < 1 || tid >= n || !(s_anc[r] >> tid & 1)) return;
    const int64_t v = (int64_t)s_draft[tid] - base;
    if (v < 0 || v >= kChunk || s_draft[tid] >= p.V) return;
    uint32_t* w = reinterpret_cast<uint32_t*>(&s_path[t][v & ~3]);
    const uint32_t one = 1u << (8 * (v & 3));
    if (add) atomicAdd(w, one);
    else atomicAnd(w, ~(0xffu << (8 * (v & 3))));
  };
  if (paths) put_path(r0, 0, true);
  __syncthreads();
  bool shared_any = false;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    if (nb > 0) {
      const int at = s_entry[first - base + e * kStep];
      if (at >= 0) {
        bias[e] = p.bias_values[b0 + at];
        shared_any = true;
      }
    }
    shared_any = shared_any || cnt[e];
  }

  for (int r = r0, t = 0; r < r1; ++r, t = t == 2 ? 0 : t + 1) {
    if (r + 1 < r1) {
      load(r + 1, nx, &nbits);
      if (paths) put_path(r + 1, t == 2 ? 0 : t + 1, true);
    }
    if (paths && r > r0) put_path(r - 1, t == 0 ? 2 : t - 1, false);
    unsigned pw[kPer];
    bool any = shared_any;
#pragma unroll
    for (int e = 0; e < kPer; ++e) pw[e] = 0;
    if (paths) {
      if (VEC) {
        const uint2 w = *reinterpret_cast<const uint2*>(&s_path[t][first - base]);
        any = any || w.x || w.y;
#pragma unroll
        for (int e = 0; e < kPer; ++e) pw[e] = (e < 4 ? w.x : w.y) >> (8 * (e & 3)) & 0xffu;
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          pw[e] = s_path[t][first - base + e * 32];
          any = any || pw[e];
        }
      }
    }
    if (any) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float f = BF16 ? __uint_as_float((uint32_t)x[e] << 16) : __uint_as_float((uint32_t)x[e]);
        const float y = steer(f, cnt[e], pw[e], rho, phi, pi, bias[e]);
        if (BF16) x[e] = (T)(pack_bf16(y, 0.f) & 0xffffu);
        else x[e] = (T)__float_as_uint(y);
      }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (!(bits >> e & 1u)) x[e] = kMinusInf;
    T* dst = reinterpret_cast<T*>(p.out) + (int64_t)(o0 + r) * p.V + first;
    if (VEC) {
      if (first < p.V) {
        reinterpret_cast<uint4*>(dst)[0] = reinterpret_cast<const uint4*>(x)[0];
        if (!BF16) reinterpret_cast<uint4*>(dst)[1] = reinterpret_cast<const uint4*>(x)[BF16 ? 0 : 1];
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (first + e * 32 < p.V) dst[e * 32] = x[e];
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = nx[e];
    bits = nbits;
    if (paths) __syncthreads();
  }
}

struct CountParams {
  const int32_t* tokens;
  const int32_t* offsets;
  uint16_t* counts;
  int32_t* status;
  int64_t n;                 // tokens in all, or (no offsets) of a sequence
  int V, parts, prompt;
};

// Prompt tokens set a bit, from as many CTAs a sequence as the host asks for.
// Emitted ones are counted by one CTA a sequence: equal tokens of a warp are
// added together, so at most eight warps meet on a word, and the sum stays at
// 32767.
__global__ void __launch_bounds__(kThreads) counts_kernel(const __grid_constant__ CountParams p) {
  dep_wait();
  dep_launch();
  const int b = blockIdx.x / p.parts, part = blockIdx.x % p.parts, lane = threadIdx.x & 31;
  int64_t a = (int64_t)b * p.n, e = a + p.n;
  if (p.offsets) {
    a = p.offsets[b];
    e = p.offsets[b + 1];
    if (a < 0 || e < a || e > p.n) {
      if (threadIdx.x == 0) set_status(p.status, TV_DEV_BAD_OFFSETS);
      return;
    }
  }
  uint32_t* row = reinterpret_cast<uint32_t*>(p.counts + (int64_t)b * ((p.V + 7) / 8 * 8));
  for (int64_t i0 = a + (int64_t)part * kThreads + (threadIdx.x & ~31); i0 < e; i0 += (int64_t)p.parts * kThreads) {
    const int64_t i = i0 + lane;
    int t = i < e ? p.tokens[i] : -1;
    if (t >= p.V) {
      set_status(p.status, TV_DEV_BAD_TOKEN);
      t = -1;
    }
    const int sh = 16 * (t & 1);
    if (p.prompt) {
      if (t >= 0) atomicOr(row + t / 2, 0x8000u << sh);
      continue;
    }
    const unsigned same = __match_any_sync(0xffffffffu, t);
    if (t < 0 || lane != __ffs(same) - 1) continue;
    const unsigned add = __popc(same);
    uint32_t old = row[t / 2];
    while (true) {
      const uint32_t have = old >> sh & 0x7fffu, now = min(have + add, 0x7fffu);
      const uint32_t want = (old & ~(0x7fffu << sh)) | now << sh;
      if (want == old) break;
      const uint32_t seen = atomicCAS(row + t / 2, old, want);
      if (seen == old) break;
      old = seen;
    }
  }
}

int check_counts_shape(const tv_logits_desc* d) {
  if (!d) return TV_ERR_NULL;
  if (d->batch < 1 || d->vocab < 1 || d->vocab > (1 << 30)) return TV_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(d->batch, align_up(d->vocab, 8), &t) || !mul_ok(t, 2, &t)) return TV_ERR_OVERFLOW;
  return TV_OK;
}

}  // namespace
}  // namespace tv

using namespace tv;

extern "C" {

int tv_token_counts_add(const tv_logits_desc* desc, const int32_t* d_tokens, const int32_t* d_offsets,
                        int64_t tokens, int32_t prompt, uint16_t* d_counts, int32_t* d_status, void* stream) {
  const int rc = check_counts_shape(desc);
  if (rc) return rc;
  if (tokens < 0 || tokens > ((int64_t)1 << 31) - 1) return TV_ERR_SHAPE;
  if (tokens == 0) return TV_OK;
  if (!d_tokens || !d_counts || !d_status) return TV_ERR_NULL;
  const void* all[] = {d_tokens, d_offsets, d_counts, d_status};
  for (const void* x : all)
    if (!aligned16(x)) return TV_ERR_ALIGN;
  CountParams p = {d_tokens, d_offsets, d_counts, d_status, tokens, desc->vocab, 1, prompt != 0};
  // prompts: about four waves of CTAs at most, each with 1024 tokens or more
  int64_t parts = prompt ? (tokens + 1023) / 1024 : 1;
  const int64_t most = (int64_t)num_sms() * 8 / desc->batch;
  if (parts > most) parts = most;
  if (parts < 1) parts = 1;
  p.parts = (int)parts;
  if (parts * desc->batch > ((int64_t)1 << 31) - 1) return TV_ERR_OVERFLOW;
  return launch_dep(counts_kernel, dim3((unsigned)(parts * desc->batch)), dim3(kThreads), 0, as_stream(stream), p) ==
                 cudaSuccess
             ? TV_OK
             : TV_ERR_CUDA;
}

int tv_tree_logits_process(const tv_logits_desc* desc, const void* d_logits, const uint16_t* d_counts,
                           const float* d_penalties, const int32_t* d_bias_offsets, const int32_t* d_bias_tokens,
                           const float* d_bias_values, const uint32_t* d_mask, const int32_t* d_draft_tokens,
                           const int32_t* d_node_offsets, const uint64_t* d_anc, void* d_out, int32_t* d_status,
                           void* stream) {
  int rc = check_counts_shape(desc);
  if (rc) return rc;
  if (desc->logits_dtype != TV_F32 && desc->logits_dtype != TV_BF16) return TV_ERR_DTYPE;
  if (desc->max_nodes < 1 || desc->max_nodes > kMaxNodes || desc->total_rows < desc->batch ||
      (int64_t)desc->total_rows > (int64_t)desc->batch * desc->max_nodes)
    return TV_ERR_TREE;
  if (d_bias_offsets && desc->biases < 0) return TV_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(desc->total_rows, desc->vocab, &t) || !mul_ok(t, 4, &t)) return TV_ERR_OVERFLOW;
  if (!d_logits || !d_node_offsets || !d_out || !d_status || !d_counts != !d_penalties ||
      !d_bias_offsets != !d_bias_tokens || !d_bias_offsets != !d_bias_values || !d_draft_tokens != !d_anc)
    return TV_ERR_NULL;
  const void* all[] = {d_logits, d_counts, d_penalties,    d_bias_offsets, d_bias_tokens, d_bias_values,
                       d_mask,   d_anc,    d_draft_tokens, d_node_offsets, d_out,         d_status};
  for (const void* x : all)
    if (!aligned16(x)) return TV_ERR_ALIGN;
  LogitsParams p = {};
  p.in = d_logits; p.out = d_out;
  p.counts = d_counts; p.penalties = d_penalties;
  p.bias_offsets = d_bias_offsets; p.bias_tokens = d_bias_tokens; p.bias_values = d_bias_values;
  p.mask = d_mask; p.draft = d_draft_tokens; p.node_offsets = d_node_offsets; p.anc = d_anc; p.status = d_status;
  p.B = desc->batch; p.V = desc->vocab; p.R = desc->total_rows; p.max_nodes = desc->max_nodes;
  p.biases = desc->biases;
  p.chunks = (desc->vocab + kChunk - 1) / kChunk;
  // rows a CTA walks: as many as leave about eight CTAs an SM, up to eight
  int64_t rows = (int64_t)desc->total_rows * p.chunks / ((int64_t)num_sms() * 8);
  rows = rows < 1 ? 1 : (rows > 8 ? 8 : rows);
  p.group_rows = (int)rows;
  p.groups = (desc->max_nodes + p.group_rows - 1) / p.group_rows;
  const int64_t grid = (int64_t)p.chunks * p.groups * p.B;
  if (grid > ((int64_t)1 << 31) - 1) return TV_ERR_OVERFLOW;
  const cudaStream_t s = as_stream(stream);
  const bool vec = desc->vocab % 8 == 0, bf = desc->logits_dtype == TV_BF16;
  const dim3 g((unsigned)grid), blk(kThreads);
  const cudaError_t e = bf ? (vec ? launch_dep(logits_kernel<true, true>, g, blk, 0, s, p)
                                  : launch_dep(logits_kernel<true, false>, g, blk, 0, s, p))
                           : (vec ? launch_dep(logits_kernel<false, true>, g, blk, 0, s, p)
                                  : launch_dep(logits_kernel<false, false>, g, blk, 0, s, p));
  return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // extern "C"
