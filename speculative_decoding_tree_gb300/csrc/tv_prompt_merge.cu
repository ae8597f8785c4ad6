#include "tv_prompt.cuh"

namespace tv {
namespace {

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

}  // namespace

cudaError_t launch_prompt_merge(const PromptParams& p, cudaStream_t s) {
  const int64_t blocks = (p.rows * p.Hq + kMergeWarps - 1) / kMergeWarps;
  const dim3 grid((unsigned)blocks), block(32 * kMergeWarps);
  if (p.d == 128) return launch_dep(prompt_merge_kernel<128>, grid, block, 0, s, p);
  if (p.d == 256) return launch_dep(prompt_merge_kernel<256>, grid, block, 0, s, p);
  return launch_dep(prompt_merge_kernel<512>, grid, block, 0, s, p);
}

}  // namespace tv
