// Causal prompt attention on the CUDA cores (fp32, and head groups the tensor
// cores' tiles do not take), and the merge of split rows.
//
// One CTA of 256 threads takes a unit of 64 query rows and walks its keys 64
// at a time with the running maximum and sum of the softmax: S = Q K^T in 4 x
// 4 blocks per thread, weights through shared memory, O += P V in registers
// (4 rows x d / 16 values per thread), all products in packed pairs.  K and V
// come in pieces of 8 KB through two shared buffers, the next piece held in
// registers while the present one is multiplied; the 64 keys' places are found
// once a step.  64 rows and 8 KB leave room for two CTAs an SM up to head_dim
// 256, whose barriers then overlap.  Bound by the fp32 units and the shared
// memory reads that feed them.
#include "tv_f32x2.cuh"
#include "tv_prompt.cuh"

namespace tv {
namespace {

constexpr int kThreads = 256;
constexpr int RPT = 4;                              // rows per thread
constexpr int BM = 16 * RPT;
constexpr int BN = 64;                              // keys a step
constexpr int KD = 32;                              // channels of a K piece
constexpr int kPiece = BN * KD;                     // floats of a piece of K or V

template <int D>
struct SCfg {
  static constexpr int QS = D + 4;                  // row strides, padded against bank conflicts
  static constexpr int PS = BN + 4;
  static constexpr int KS = KD + 4;
  static constexpr int VK = kPiece / D;             // keys of a V piece
  static constexpr int BUF = BN * KS;               // floats of a buffer (K's padded piece is the larger)
  static constexpr int SMEM = (BM * QS + BM * PS + 2 * BUF) * 4;
  static constexpr int OC = D / 64;                 // groups of four columns per thread
};

template <bool BF16>
__device__ __forceinline__ float4 load4(const void* base, int64_t elem) {
  if (BF16) {
    const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(base) + elem);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
  }
  return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + elem);
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, D == 512 ? 1 : 2)
prompt_simt_kernel(const __grid_constant__ PromptParams p) {
  using C = SCfg<D>;
  constexpr int OC = C::OC;
  extern __shared__ __align__(16) float smem[];
  float* sQ = smem;
  float* sP = sQ + BM * C::QS;
  float* sB = sP + BM * C::PS;
  __shared__ int64_t s_at[2][BN];                   // first element of a step's keys, -1: none (zeros)
  __shared__ int s_b, s_i, s_bad;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  dep_wait();
  dep_launch();
  const int s = blockIdx.x % p.splits;
  const int rest = blockIdx.x / p.splits;
  const int g = rest % p.Hkv;
  if (tid < 32) {
    int b = -1, i = 0;
    if (!find_unit(p, rest / p.Hkv, &b, &i)) b = -1;
    if (tid == 0) {
      s_b = b;
      s_i = i;
      s_bad = 0;
    }
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;
  int64_t o0, n;
  prompt_rows(p.row_offsets, b, p.rows, p.max_rows, p.status, &o0, &n);
  const int64_t Praw = p.prefix_len[b], P = clamp_prefix(Praw, p.max_prefix, p.capacity);
  if (P != Praw && tid == 0) set_status(p.status, TV_DEV_BAD_PREFIX);
  const int64_t m0 = (int64_t)s_i * BM, nrows = n * p.G;
  const int64_t mlast = min(nrows, m0 + BM) - 1;
  const int Pt = (int)((P + kPromptTile - 1) / kPromptTile);
  const int t_begin = s * p.chunk_tiles;
  const int t_end = min(Pt + (int)(mlast / p.G / kPromptTile) + 1, t_begin + p.chunk_tiles);
  if (t_begin >= t_end) return;
  // steps of 64 keys; the last may lie past every row's keys
  const int step0 = t_begin * 2, psteps = Pt * 2;
  int step1 = t_end * 2;
  if (t_end > Pt && mlast / p.G - (int64_t)(t_end - 1 - Pt) * kPromptTile < BN) --step1;

  // places of step st's keys
  auto find_keys = [&](int st) {
    if (tid >= BN) return;
    const int64_t key = (int64_t)(st < psteps ? st : st - psteps) * BN + tid;
    int64_t at = -1;
    if (st >= psteps) {
      if (key < n) at = ((int64_t)g * p.rows + o0 + key) * D;
    } else if (key < P) {
      if (!p.paged) {
        at = (((int64_t)b * p.Hkv + g) * p.capacity + key) * D;
      } else {
        const int pid = p.page_table[(int64_t)b * p.max_pages + key / kPageSize];
        if (pid >= 0 && pid < p.num_pages) at = (((int64_t)pid * p.Hkv + g) * kPageSize + key % kPageSize) * D;
        else s_bad = 1;
      }
    }
    s_at[st & 1][tid] = at;
  };
  find_keys(step0);
  for (int e = tid; e < BM * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    float4 v = make_float4(0, 0, 0, 0);
    if (m0 + r < nrows)
      v = load4<BF16>(p.q, ((o0 + (m0 + r) / p.G) * p.Hq + g * p.G + (m0 + r) % p.G) * D + c);
    *reinterpret_cast<float4*>(sQ + r * C::QS + c) = v;
  }
  int seen[RPT];                                    // own rows this row sees: 0 .. seen
#pragma unroll
  for (int i = 0; i < RPT; ++i) seen[i] = (int)(min(m0 + ty * RPT + i, nrows - 1) / p.G);
  __syncthreads();

  // piece c of step st: K pieces 0 .. D / 32 - 1 (64 keys x 32 channels), then V pieces (VK keys x D)
  constexpr int KP = D / KD, NP = KP + BN / C::VK;
  float4 hold[2];
  auto fetch = [&](int st, int c) {
    const bool own = st >= psteps, isk = c < KP;
    const void* src = isk ? (own ? p.k_rows : p.k_cache) : (own ? p.v_rows : p.v_cache);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int f = (tid + e * kThreads) * 4;       // of the piece's 2048 floats
      const int j = isk ? f / KD : (c - KP) * C::VK + f / D;
      const int ch = isk ? c * KD + f % KD : f % D;
      const int64_t at = s_at[st & 1][j];
      hold[e] = at < 0 ? make_float4(0, 0, 0, 0) : load4<BF16>(src, at + ch);
    }
  };
  auto put = [&](int c, float* buf) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int f = (tid + e * kThreads) * 4;
      *reinterpret_cast<float4*>(buf + (c < KP ? f / KD * C::KS + f % KD : f)) = hold[e];
    }
  };

  uint64_t o[RPT][OC][2];                           // pairs of columns
  float m_run[RPT], l_run[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
#pragma unroll
    for (int c = 0; c < OC; ++c) o[i][c][0] = o[i][c][1] = 0ull;
  }
  int par = 0;
  fetch(step0, 0);
  for (int st = step0; st < step1; ++st) {
    if (st + 1 < step1) find_keys(st + 1);          // seen by the others after the next barrier
    uint64_t sc[RPT][4];                            // sums of the even and of the odd channels
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[i][j] = 0ull;
#pragma unroll 1
    for (int c = 0; c < KP; ++c) {
      float* buf = sB + par * C::BUF;
      par ^= 1;
      put(c, buf);
      __syncthreads();
      fetch(st, c + 1);
#pragma unroll
      for (int k = 0; k < KD; k += 4) {
        ulonglong2 kv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(buf + (tx + 16 * j) * C::KS + k);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(sQ + (ty * RPT + i) * C::QS + c * KD + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[i][j] = ffma2(qv.y, kv[j].y, ffma2(qv.x, kv[j].x, sc[i][j]));
        }
      }
    }
    // mask, running maximum and sum; a row's 64 scores lie with the 16 threads of its half warp
    const bool own = st >= psteps;
    const int64_t j0 = (int64_t)(own ? st - psteps : st) * BN;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int64_t lim = (own ? (int64_t)seen[i] : P - 1) - j0 - tx;   // keys 16 j up to here are seen
      float x[4], mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = up2(sc[i][j]);
        x[j] = 16 * j <= lim ? (v.x + v.y) * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, x[j]);
      }
#pragma unroll
      for (int a = 8; a > 0; a >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, a));
      const float m_new = fmaxf(m_run[i], mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m_run[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = exp2f(x[j] - ref);
        sum += w;
        sP[(ty * RPT + i) * C::PS + tx + 16 * j] = w;
      }
#pragma unroll
      for (int a = 8; a > 0; a >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, a);
      l_run[i] = l_run[i] * alpha + sum;
      m_run[i] = m_new;
      const uint64_t a2 = pk2(alpha, alpha);
#pragma unroll
      for (int c = 0; c < OC; ++c) {
        o[i][c][0] = ffma2(o[i][c][0], a2, 0ull);
        o[i][c][1] = ffma2(o[i][c][1], a2, 0ull);
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int c = KP; c < NP; ++c) {
      float* buf = sB + par * C::BUF;
      par ^= 1;
      put(c, buf);
      __syncthreads();
      if (c + 1 < NP) fetch(st, c + 1);
      else if (st + 1 < step1) fetch(st + 1, 0);
      const int k0 = (c - KP) * C::VK;
#pragma unroll(C::VK > 8 ? 2 : 1)
      for (int k = 0; k < C::VK; k += 4) {
        float4 w[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          w[i] = *reinterpret_cast<const float4*>(sP + (ty * RPT + i) * C::PS + k0 + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint64_t w2[RPT];
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float x = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
            w2[i] = pk2(x, x);
          }
#pragma unroll
          for (int c4 = 0; c4 < OC; ++c4) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(buf + (k + kk) * D + tx * 4 + 64 * c4);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              o[i][c4][0] = ffma2(w2[i], v.x, o[i][c4][0]);
              o[i][c4][1] = ffma2(w2[i], v.y, o[i][c4][1]);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t m = m0 + ty * RPT + i;
    if (m >= nrows) continue;
    const int64_t row = o0 + m / p.G;
    const int h = g * p.G + (int)(m % p.G);
    const float inv = l_run[i] > 0.f ? 1.f / l_run[i] : (l_run[i] == 0.f ? 0.f : l_run[i]);
    const int my_s = (Pt + seen[i] / kPromptTile) / p.chunk_tiles;   // the row's last split
    if (s > my_s) continue;
    const bool split = my_s > 0;
    const int64_t slot = split ? prompt_slot(row, h, s, p.Hq, p.splits) : row * p.Hq + h;
#pragma unroll
    for (int c4 = 0; c4 < OC; ++c4) {
      const float2 lo = up2(o[i][c4][0]), hi = up2(o[i][c4][1]);
      const float4 v = make_float4(lo.x * inv, lo.y * inv, hi.x * inv, hi.y * inv);
      const int64_t at = slot * D + tx * 4 + 64 * c4;
      if (split) *reinterpret_cast<float4*>(p.o_part + at) = v;
      else if (p.out_bf16)
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
      else *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) = v;
    }
    if (split && tx == 0) p.ml_part[slot] = make_float2(m_run[i], l_run[i]);
  }
  __syncthreads();
  if (tid == 0 && s_bad) set_status(p.status, TV_DEV_BAD_PAGE);
}

// The rows that two splits or more attended to: out = sum_s w_s O_s with
// w_s = l_s 2^(m_s - M) / L.  One warp a (row, head); bound by the partials'
// reads, which are still in L2.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prompt_merge_kernel(const __grid_constant__ PromptParams p) {
  dep_wait();
  dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int64_t row = w / p.Hq;
  const int h = (int)(w - row * p.Hq);
  if (row >= p.rows) return;
  // the row's sequence: the last one that starts at or before it
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.row_offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  int64_t o0, n;
  if (!prompt_rows(p.row_offsets, lo, p.rows, p.max_rows, p.status, &o0, &n) || row < o0 || row >= o0 + n) return;
  const int64_t P = clamp_prefix(p.prefix_len[lo], p.max_prefix, p.capacity);
  const int64_t tile = (P + kPromptTile - 1) / kPromptTile + (row - o0) / kPromptTile;
  const int ns = (int)(tile / p.chunk_tiles) + 1;
  if (ns < 2) return;
  const int64_t slot = prompt_slot(row, h, 0, p.Hq, p.splits);
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, p.ml_part[slot + s].x);
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 acc[D / 128];
#pragma unroll
  for (int c = 0; c < D / 128; ++c) acc[c] = make_float4(0, 0, 0, 0);
#pragma unroll 2
  for (int s = 0; s < ns; ++s) {
    const float2 ml = p.ml_part[slot + s];
    const float wt = ml.y * exp2f(ml.x - ref);
    L += wt;
    if (wt == 0.f) continue;                        // a split whose keys this row does not see
    const float4* src = reinterpret_cast<const float4*>(p.o_part + (slot + s) * D) + lane;
#pragma unroll
    for (int c = 0; c < D / 128; ++c) {
      const float4 v = src[c * 32];
      acc[c].x = fmaf(wt, v.x, acc[c].x);
      acc[c].y = fmaf(wt, v.y, acc[c].y);
      acc[c].z = fmaf(wt, v.z, acc[c].z);
      acc[c].w = fmaf(wt, v.w, acc[c].w);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int c = 0; c < D / 128; ++c) {
    const int64_t at = (row * p.Hq + h) * D + lane * 4 + c * 128;
    const float4 v = make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
    if (p.out_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at) =
          make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    else *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) = v;
  }
}

template <bool BF16, int D>
cudaError_t launch_d(const PromptParams& p, int64_t units, cudaStream_t s) {
  const cudaError_t e = ensure_max_dynamic_smem<prompt_simt_kernel<BF16, D>>(SCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dep(prompt_simt_kernel<BF16, D>, dim3((unsigned)(units * p.Hkv * p.splits)), dim3(kThreads),
                    SCfg<D>::SMEM, s, p);
}

}  // namespace

int prompt_simt_rows() { return BM; }
int prompt_simt_ctas_per_sm(int d) { return d == 512 ? 1 : 2; }

cudaError_t launch_prompt_simt(const PromptParams& p, int dtype, int64_t units, cudaStream_t s) {
  const bool bf = dtype == TV_BF16;
  if (p.d == 128) return bf ? launch_d<true, 128>(p, units, s) : launch_d<false, 128>(p, units, s);
  if (p.d == 256) return bf ? launch_d<true, 256>(p, units, s) : launch_d<false, 256>(p, units, s);
  return bf ? launch_d<true, 512>(p, units, s) : launch_d<false, 512>(p, units, s);
}

cudaError_t launch_prompt_merge(const PromptParams& p, cudaStream_t s) {
  const int64_t blocks = (p.rows * p.Hq + kMergeWarps - 1) / kMergeWarps;
  const dim3 grid((unsigned)blocks), block(32 * kMergeWarps);
  if (p.d == 128) return launch_dep(prompt_merge_kernel<128>, grid, block, 0, s, p);
  if (p.d == 256) return launch_dep(prompt_merge_kernel<256>, grid, block, 0, s, p);
  return launch_dep(prompt_merge_kernel<512>, grid, block, 0, s, p);
}

}  // namespace tv
