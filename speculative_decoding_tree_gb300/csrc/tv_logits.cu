// The control of tree logits (include/tree_logits.h): penalties, biases and
// grammar masks on every tree row, and the token counts they read.
//
// process: a CTA takes 2048 logits of up to 8 tree rows of one sequence.  Few
// tokens are counted, biased or on a row's path, so the work is two passes.
// The first masks and copies: a thread 8 neighbours of each row on a 16-byte
// boundary of memory (a vocabulary's rows start anywhere: they stand for the
// tokens from 8 k - a on, a = row * vocab mod 8), the loads of four rows
// (fp32: two) under way at once, and 8 logits that the mask forbids altogether are
// not read.  Meanwhile the CTA lists the tokens of its chunk that the rows
// share something of, and the drafts on each row's path.  The second pass
// takes (row, listed token) pairs, one a thread, and recomputes those logits
// in place: a forbidden one is -inf by then and stays, an allowed one is
// still the input.  One pass that looked at every logit's tables as it passed
// took three times the instructions (16 trees 126 - 227 us, now 72).  Bound by the
// bytes.
#include "tree_logits.h"
#include "tv_host.cuh"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                             // tokens a thread
constexpr int kChunk = kThreads * kPer;
constexpr int kRows = 8;                            // rows a CTA, at most
constexpr int kSpan = kChunk + 8;                   // tokens a CTA's logits may stand for: base - 8 .. base + 2047
constexpr int kTouch = kSpan / 32 + 2;              // words of their bits, and one to read past the end

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

template <bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 6) logits_kernel(const __grid_constant__ LogitsParams p) {
  constexpr int W = BF16 ? 4 : 8;                   // 32-bit words of 8 logits
  constexpr int U = BF16 ? 4 : 2;                   // rows under way
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ uint32_t s_shared[kTouch];             // a bit a token: counted or biased,
  __shared__ uint32_t s_biased[kTouch];             // biased,
  __shared__ uint32_t s_drafts[kRows][kTouch];      // a draft on the row's path
  __shared__ uint32_t s_tokens[kSpan];              // the tokens of s_shared: place, and count word << 16
  __shared__ int s_entry[kSpan];                    // of the biased tokens: the list's entry
  __shared__ uint16_t s_path[kRows][64], s_once[kRows][64];   // places of the path's drafts, and those of them that
                                                    // are not in s_shared, once each
  __shared__ int s_ntokens, s_npath[kRows], s_nonce[kRows];
  const int tid = threadIdx.x;
  dep_wait();
  dep_launch();
  const int c = blockIdx.x % p.chunks;
  const int grp = blockIdx.x / p.chunks % p.groups;
  const int b = blockIdx.x / p.chunks / p.groups;
  int o0, n;
  if (!seq_rows(p.node_offsets, b, p.R, p.max_nodes, p.status, &o0, &n)) return;
  const int r0 = grp * p.group_rows, nr = min(n - r0, p.group_rows);
  if (nr <= 0) return;
  const int base = c * kChunk;                      // (V <= 2^30)
  const int words = (p.V + 31) / 32;
  const int64_t row0 = o0 + r0;
  const bool counted = p.counts != nullptr, paths = counted && p.draft != nullptr;

  // ---------------------------------------------------------------- first pass: loads
  auto shift = [&](int i) { return ALIGNED ? 0 : (int)((row0 + i) * p.V & 7); };
  auto first_token = [&](int i) { return base + tid * kPer - shift(i); };
  uint32_t allow[kRows / 4];                        // the mask's bits, 8 a row
#pragma unroll
  for (int i = 0; i < kRows / 4; ++i) allow[i] = p.mask ? 0u : 0xffffffffu;
  if (p.mask) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int t = first_token(i);
      if (i >= nr || t >= p.V || t <= -kPer) continue;
      const uint32_t* row = p.mask + (row0 + i) * words;
      uint32_t m;
      if (ALIGNED) {
        m = reinterpret_cast<const uint8_t*>(row)[t >> 3];
      } else {
        const int w = t >> 5, sh = t & 31;          // (t may be -7 .. -1: word -1 has no token)
        const uint32_t lo = w >= 0 ? row[w] : 0u, hi = sh > 24 && w + 1 < words ? row[w + 1] : 0u;
        m = __funnelshift_r(lo, hi, sh) & 0xffu;
      }
      allow[i / 4] |= m << (8 * (i & 3));
    }
  }
  auto mask_of = [&](int i) { return allow[i / 4] >> (8 * (i & 3)) & 0xffu; };
  uint32_t x[U][W];
  auto load = [&](int i, uint32_t (&d)[W]) {
    const int t = first_token(i);
    if (i >= nr || mask_of(i) == 0 || t >= p.V || t <= -kPer) return;
    const char* src = reinterpret_cast<const char*>(p.in) + ((row0 + i) * p.V + t) * ES;
    if (ALIGNED || (t >= 0 && t + kPer <= p.V)) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const uint4 v = reinterpret_cast<const uint4*>(src)[q];
        d[4 * q] = v.x;
        d[4 * q + 1] = v.y;
        d[4 * q + 2] = v.z;
        d[4 * q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const bool in = t + e >= 0 && t + e < p.V;
        if (BF16) {
          const uint32_t v = in ? reinterpret_cast<const uint16_t*>(src)[e] : 0u;
          d[BF16 ? e / 2 : e] = e & 1 ? d[BF16 ? e / 2 : e] | v << 16 : v;
        } else {
          d[BF16 ? 0 : e] = in ? reinterpret_cast<const uint32_t*>(src)[e] : 0u;
        }
      }
    }
  };
  auto store = [&](int i, uint32_t (&d)[W]) {
    const int t = first_token(i);
    if (i >= nr || t >= p.V || t <= -kPer) return;
    const uint32_t m = mask_of(i);
    if (m != 0xffu) {
#pragma unroll
      for (int q = 0; q < W; ++q) {
        if (BF16) {
          const uint32_t two = m >> (2 * q) & 3u, keep = ((two | two << 15) & 0x00010001u) * 0xffffu;
          d[q] = (d[q] & keep) | (0xff80ff80u & ~keep);
        } else if (!(m >> q & 1u)) {
          d[q] = 0xff800000u;
        }
      }
    }
    char* dst = reinterpret_cast<char*>(p.out) + ((row0 + i) * p.V + t) * ES;
    if (ALIGNED || (t >= 0 && t + kPer <= p.V)) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q)
        reinterpret_cast<uint4*>(dst)[q] = make_uint4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (t + e < 0 || t + e >= p.V) continue;
        if (BF16) reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(d[BF16 ? e / 2 : e] >> (16 * (e & 1)));
        else reinterpret_cast<uint32_t*>(dst)[e] = d[BF16 ? 0 : e];
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, x[u]);

  // ---------------------------------------------------------------- the lists
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
  const bool any = counted || nb > 0;
  float rho = 1.f, phi = 0.f, pi = 0.f;
  if (any) {
    const uint16_t* counts = p.counts + (int64_t)b * ((p.V + 7) / 8 * 8);
    if (counted) {
      rho = p.penalties[b * 3];
      phi = p.penalties[b * 3 + 1];
      pi = p.penalties[b * 3 + 2];
    }
    // this thread's places 8 tid .. 8 tid + 7, i.e. tokens from base - 8 + 8 tid on; the last 8 are thread 0's
    auto count_words = [&](int e) {
      const int t = base - 8 + e * 8;
      return counted && e < kSpan / 8 && t >= 0 && t < p.V ? *reinterpret_cast<const uint4*>(counts + t)
                                                           : make_uint4(0, 0, 0, 0);
    };
    const uint4 w0 = count_words(tid), w1 = tid == 0 ? count_words(kThreads) : make_uint4(0, 0, 0, 0);
    for (int e = tid; e < nr * kTouch; e += kThreads) (&s_drafts[0][0])[e] = 0;
    for (int e = tid; e < kTouch; e += kThreads) s_biased[e] = 0;
    if (tid < kRows) s_npath[tid] = s_nonce[tid] = 0;
    if (tid == 0) s_ntokens = 0;
    // the biased tokens of the chunk: entry -1 first, then the largest number
    auto biased = [&](int e) {
      const int t = p.bias_tokens[b0 + e];
      if ((unsigned)t >= (unsigned)p.V) {
        if (c == 0) set_status(p.status, TV_DEV_BAD_TOKEN);
        return -1;
      }
      return t >= base - 8 && t < base + kChunk ? t - base + 8 : -1;
    };
    for (int e = tid; e < nb; e += kThreads) {
      const int at = biased(e);
      if (at >= 0) s_entry[at] = -1;
    }
    __syncthreads();
    for (int e = tid; e < nb; e += kThreads) {
      const int at = biased(e);
      if (at >= 0) {
        atomicMax(&s_entry[at], e);
        atomicOr(&s_biased[at >> 5], 1u << (at & 31));
      }
    }
    __syncthreads();
    auto list = [&](int e, const uint4& w) {        // the 8 places of byte e
      uint32_t bits = reinterpret_cast<const uint8_t*>(s_biased)[e];
      const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) bits |= (a[q] & 0xffffu ? 1u : 0u) << (2 * q) | (a[q] >> 16 ? 2u : 0u) << (2 * q);
      reinterpret_cast<uint8_t*>(s_shared)[e] = (uint8_t)bits;
      if (!bits) return;
      int k = atomicAdd(&s_ntokens, __popc(bits));
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (bits >> q & 1u) s_tokens[k++] = (uint32_t)(e * 8 + q) | (a[q / 2] >> (16 * (q & 1))) << 16;
    };
    list(tid, w0);
    if (tid == 0) list(kThreads, w1);
    if (paths) {
      __syncthreads();
      for (int e = tid; e < nr * 64; e += kThreads) {
        const int i = e >> 6, j = e & 63;
        if (j < 1 || j >= n || !(p.anc[row0 + i] >> j & 1)) continue;
        const int t = p.draft[o0 + j];
        if ((unsigned)t >= (unsigned)p.V || t < base - 8 || t >= base + kChunk) continue;
        const int at = t - base + 8;
        const uint32_t bit = 1u << (at & 31);
        s_path[i][atomicAdd(&s_npath[i], 1)] = (uint16_t)at;   // (in any order: they are only counted)
        const bool seen = atomicOr(&s_drafts[i][at >> 5], bit) & bit;
        if (!seen && !(s_shared[at >> 5] & bit)) s_once[i][atomicAdd(&s_nonce[i], 1)] = (uint16_t)at;
      }
    }
  }

  // ---------------------------------------------------------------- first pass: stores
#pragma unroll
  for (int i0 = 0; i0 < kRows; i0 += U) {
    if (i0 >= nr) break;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 > 0) load(i0 + u, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) store(i0 + u, x[u]);
  }
  if (!any) return;
  __syncthreads();

  // ---------------------------------------------------------------- second pass: the listed tokens
  auto fix = [&](int i, int at, uint32_t word) {
    const int t = base - 8 + at, mine = at - 8 + shift(i);
    if (mine < 0 || mine >= kChunk || t < 0 || t >= p.V) return;   // another CTA's, in this row
    char* dst = reinterpret_cast<char*>(p.out) + ((row0 + i) * p.V + t) * ES;
    const float f = BF16 ? __uint_as_float((uint32_t)*reinterpret_cast<uint16_t*>(dst) << 16)
                         : *reinterpret_cast<float*>(dst);
    if (f == -INFINITY) return;
    const uint32_t bit = 1u << (at & 31);
    unsigned on = 0;                                // drafts of the path that are this token
    if (paths && (s_drafts[i][at >> 5] & bit))
      for (int k = 0; k < s_npath[i]; ++k) on += s_path[i][k] == at;
    const float bias = nb > 0 && (s_biased[at >> 5] & bit) ? p.bias_values[b0 + s_entry[at]] : 0.f;
    const float y = steer(f, word, on, rho, phi, pi, bias);
    if (BF16) *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(y);
    else *reinterpret_cast<float*>(dst) = y;
  };
  const int nt = s_ntokens;
  for (int e = tid; e < nt * nr; e += kThreads) {
    const int i = e / nt;
    const uint32_t w = s_tokens[e - i * nt];
    fix(i, (int)(w & 0xffffu), w >> 16);
  }
  if (paths) {
    for (int e = tid; e < nr * 64; e += kThreads)
      if ((e & 63) < s_nonce[e >> 6]) fix(e >> 6, s_once[e >> 6][e & 63], 0u);
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
  const bool aligned = desc->vocab % 8 == 0;
  p.chunks = (desc->vocab + (aligned ? 0 : 7) + kChunk - 1) / kChunk;   // a row may start 7 logits into its first 8
  // rows a CTA takes: as many as leave about four CTAs an SM
  int64_t rows = (int64_t)desc->total_rows * p.chunks / ((int64_t)num_sms() * 4);
  rows = rows < 1 ? 1 : (rows > kRows ? kRows : rows);
  p.group_rows = (int)rows;
  p.groups = (desc->max_nodes + p.group_rows - 1) / p.group_rows;
  const int64_t grid = (int64_t)p.chunks * p.groups * p.B;
  if (grid > ((int64_t)1 << 31) - 1) return TV_ERR_OVERFLOW;
  const cudaStream_t s = as_stream(stream);
  const dim3 g((unsigned)grid), blk(kThreads);
  const bool bf = desc->logits_dtype == TV_BF16;
  const cudaError_t e = bf ? (aligned ? launch_dep(logits_kernel<true, true>, g, blk, 0, s, p)
                                      : launch_dep(logits_kernel<true, false>, g, blk, 0, s, p))
                           : (aligned ? launch_dep(logits_kernel<false, true>, g, blk, 0, s, p)
                                      : launch_dep(logits_kernel<false, false>, g, blk, 0, s, p));
  return e == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // extern "C"
