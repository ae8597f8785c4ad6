// Split-KV tree-verify attention over a 4-bit cache (tree_kv4.h) for few query
// rows: up to 8 per KV head (plain decoding, short chains), bf16 queries and
// tree K/V, fp32 accumulation and softmax.
//
// With so few rows the pass is bound by the cache's bytes, provided that the
// expansion of the codes costs little beside it: 46 values a clock and SM
// arrive at the memory's rate.  So the expanded values never leave the
// registers: a warp loads packed words from global memory straight into the
// lanes that need them, expands a word's pairs there (mask, and one fused
// multiply-add: see tv_attn_kv4.cu) and multiplies with mma.sync.m16n8k16,
// whose row granularity (8 query rows) fits where a tcgen05 operand would have
// to go through tensor memory.  64 sequences x 4 rows over up to 16384 keys:
// 152 us (the floor of its bytes is 90), 209 with tcgen05's 16-column tile.  From
// 9 rows on that tile is the faster one: 64 x 16 rows 214 us, 242 with two
// mma.sync columns here.
//
//   S^T [16 keys x 8 rows]     = K  [16 keys x 16 channels]      Q^T
//   O^T [16 channels x 8 rows] += V^T [16 channels x 16 keys]    P^T
//
// Lane (g = lane / 4, t = lane % 4) of an A operand holds rows g and g + 8 and
// two column pairs.  Which channels and keys these are is free as long as both
// operands agree, so they are chosen to make the lanes' loads whole:
// * a span is 64 keys (4 blocks).  Row r (0..15) of key tile mt (0..3) is key
//   16 (r % 8 / 2) + 2 (2 mt + r / 8) + r % 2: lane g works on block g / 2;
// * K: lane t takes channels 32 t .. 32 t + 31 of a 128-channel chunk, the 16
//   bytes of a key's group, and its one scale; each 16-byte load is 4 pairs x
//   4 words, 8 k-steps;
// * V: lane t takes the 16 keys of block t; rows g and g + 8 of channel tile ct
//   are channels 16 ct + 2 g and + 1, one 16-byte load;
// * P^T comes from S^T's registers by an 8 x 8 transpose of bf16 pairs
//   (movmatrix).
//
// The softmax's exponent reference of a row is its score with the warp's first
// key (any reference within 2^60 of the maximum gives the same weights); a
// score further above moves it.  A warp keeps its own references, sums and O;
// its CTA's four warps take alternate spans and join at the end.  Each load
// buffer is refilled as soon as it has been multiplied, a span ahead.
#include <climits>

#include "tv_kv4.cuh"

namespace tv {
namespace {

using kv4::fma_bf16x2;
using kv4::kMinus136;
using kv4::kMinusZero;
using kv4::kOne;
using kv4::PairBits;

constexpr int kSpan = 64;                        // keys per span
constexpr int kRows = 8;                         // query rows of a KV head: an mma.sync column each
constexpr int kWarps = 4;
constexpr float kHeadroom = 60.0f;               // log2: a weight above 2^60 moves the reference
constexpr int kNoPage = INT_MIN;                 // nothing to load (past the end, or seen by no row): not a page id

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// through L2: blocks of two heads share cache lines, and the kernel before
// may have written one of them
__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }

template <int D>
struct Cfg {
  static constexpr int CPT = D / 128;
  static constexpr int CTAS = D == 128 ? 3 : 2;               // per SM (registers)
  static constexpr bool QREG = D <= 256;                      // queries in registers, else in shared memory
  static constexpr int OUT_PITCH = D + 8;
  static constexpr int SMEM = kWarps * 8 * OUT_PITCH * 4 > CPT * 8 * 32 * 8 ? kWarps * 8 * OUT_PITCH * 4
                                                                                     : CPT * 8 * 32 * 8;
};

template <int D, bool WIN>
__global__ void __launch_bounds__(32 * kWarps, Cfg<D>::CTAS) tv_attn_kv4_rows_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D>;
  constexpr int CPT = C::CPT, KB = kv4::k_block_bytes(D), VB = kv4::v_block_bytes(D);
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(16) float smem[];
  __shared__ float s_m[kWarps][8], s_l[kWarps][8];
  dep_wait();
  dep_launch();
  const int g_head = blockIdx.y / p.splits, s_id = blockIdx.y % p.splits, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t Praw = p.prefix_len[b];
  int o0, n;
  if (!seq_rows(p.node_offsets, b, p.R, p.max_nodes, p.status, &o0, &n)) return;
  const int live = n * p.G;                        // rows of this sequence, kRows at most
  if (live <= 0) return;
  const int64_t P = clamp_prefix(Praw, p.max_prefix, p.capacity);
  if (P != Praw && tid == 0 && s_id == 0 && g_head == 0) set_status(p.status, TV_DEV_BAD_PREFIX);
  const KeyMap km = key_map(P, WIN ? p.window : 0, p.sinks, p.map_tile);
  const int nch = num_chunks(km.len, p.chunk, p.tree_tile);
  if (s_id >= nch) return;
  const int64_t k_begin = (int64_t)s_id * p.chunk, k_end = min(km.len, k_begin + p.chunk);
  const int nsp = k_end > k_begin ? (int)((k_end - k_begin + kSpan - 1) / kSpan) : 0;   // prefix spans
  const int total = nsp + (s_id == nch - 1 ? 1 : 0);                                    // the tree is the last one
  const int64_t first_pos = WIN ? P - p.window + 1 : 0;
  const PairBits pair;
  const uint8_t* k4 = reinterpret_cast<const uint8_t*>(p.k_cache);
  const uint8_t* v4 = reinterpret_cast<const uint8_t*>(p.v_cache);

  // element offset of query row r (node r / G, head r % G of the group) in q and out
  auto row_at = [&](int r) -> int64_t { return ((int64_t)(o0 + r / p.G) * p.Hq + g_head * p.G + r % p.G) * D; };
  // Q^T fragments: k-step j of chunk c takes channels 32 t + 8 (j / 2) + 4 (j % 2) .. + 3 of row g
  uint32_t q[C::QREG ? CPT : 1][8][2];
  uint2* sq = reinterpret_cast<uint2*>(smem);
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                                      row_at(g < live ? g : 0) + c * 128 + 32 * t);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint4 v = g < live ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
      if (C::QREG) {
        q[C::QREG ? c : 0][2 * w][0] = v.x;
        q[C::QREG ? c : 0][2 * w][1] = v.y;
        q[C::QREG ? c : 0][2 * w + 1][0] = v.z;
        q[C::QREG ? c : 0][2 * w + 1][1] = v.w;
      } else if (warp == 0) {
        sq[(c * 8 + 2 * w) * 32 + lane] = make_uint2(v.x, v.y);
        sq[(c * 8 + 2 * w + 1) * 32 + lane] = make_uint2(v.z, v.w);
      }
    }
  }
  if (!C::QREG) __syncthreads();

  // The blocks a lane reads of span sp: block g / 2 (K, and the V scales of its
  // keys) and block t (V).  Blocks past the end or seen by no row stand at
  // block 0 (their keys are masked, and every code is a finite number); a bad
  // page is flagged and its codes read as zeros.
  struct Blocks {
    int64_t k, v;
    bool bad_k, bad_v;
  };
  auto page_of = [&](int sp, int j) -> int {       // page id, or block number; kNoPage: none
    const int64_t v = k_begin + (int64_t)sp * kSpan + j * kPageSize;
    if (sp >= nsp || v >= k_end) return kNoPage;
    const int64_t pos = WIN ? km.pos(v) : v;
    if (WIN && pos >= p.sinks && pos + kPageSize <= first_pos) return kNoPage;
    // (the table may hold any number: every negative one is out of range, and -1 stands for them all)
    return p.paged ? max(p.page_table[(int64_t)b * p.max_pages + pos / kPageSize], -1) : (int)(pos / kPageSize);
  };
  auto block_of = [&](int id, bool* bad) -> int64_t {
    *bad = false;
    if (id == kNoPage) return 0;
    if (!p.paged) return ((int64_t)b * p.Hkv + g_head) * p.max_pages + id;
    if (id >= 0 && id < p.num_pages) return (int64_t)id * p.Hkv + g_head;
    *bad = true;
    set_status(p.status, TV_DEV_BAD_PAGE);
    return 0;
  };

  float o[CPT][8][4];
  float nm[2], l[2];                               // rows 2 t, 2 t + 1
  int refs = 0;                                    // references: 0 none yet, 1 of some rows, 2 of all
#pragma unroll
  for (int c = 0; c < CPT; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][i][e] = 0.f;
  nm[0] = nm[1] = 0.f;
  l[0] = l[1] = 0.f;

  // pieces of a span: K of each 128-channel chunk, then V; piece i sits in
  // buf[i & 1] and is loaded once piece i - 2 has been used
  uint4 buf[2][8], ksc[2], vsc;
  auto load_k = [&](uint4 (&r)[8], uint4& sc, const Blocks& bl, int c) {
    const uint8_t* src = k4 + bl.k * KB + (4 * c + t) * 256 + (g & 1) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = ldg16(src + i * 32);        // position 2 i + g % 2 of the block
    sc = ldg16(k4 + bl.k * KB + 8 * D + (4 * c + t) * 16);
    if (bl.bad_k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
    }
  };
  auto load_v = [&](uint4 (&r)[8], const Blocks& bl, int c) {
    const uint8_t* src = v4 + bl.v * VB + (128 * c + 2 * g) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = ldg16(src + i * 128);       // channels 16 i + 2 g, + 1
    if (bl.bad_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
    }
  };
  auto blocks = [&](int id_k, int id_v) -> Blocks {
    Blocks r;
    r.k = block_of(id_k, &r.bad_k);
    r.v = block_of(id_v, &r.bad_v);
    return r;
  };

  // S^T of one chunk from its expanded operand
  float s[4][4];
  auto qk_step = [&](int c, int j, int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    if (C::QREG) {
      mma(s[mt], a0, a1, a2, a3, q[C::QREG ? c : 0][j][0], q[C::QREG ? c : 0][j][1]);
    } else {
      const uint2 qq = sq[(c * 8 + j) * 32 + lane];
      mma(s[mt], a0, a1, a2, a3, qq.x, qq.y);
    }
  };
  auto qk = [&](const uint4 (&r)[8], const uint4& sc, int c) {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      // keys 2 (2 mt) + g % 2 and 2 (2 mt + 1) + g % 2 of the block
      uint32_t s2[2], o2[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t code = (word(sc, mt) >> (16 * h + 8 * (g & 1))) & 255u;
        s2[h] = ((code << 4) + 0x3800u) * 0x00010001u;
        o2[h] = fma_bf16x2(s2[h], kMinus136, kMinusZero);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w0 = word(r[2 * mt], j >> 1), w1 = word(r[2 * mt + 1], j >> 1);
        const int e = 2 * (j & 1);
        qk_step(c, j, mt, fma_bf16x2(pair(w0, e), s2[0], o2[0]), fma_bf16x2(pair(w1, e), s2[1], o2[1]),
                fma_bf16x2(pair(w0, e + 1), s2[0], o2[0]), fma_bf16x2(pair(w1, e + 1), s2[1], o2[1]));
      }
    }
  };
  // the position in the span of key tile mt, half h, for this lane's row g
  auto key_of = [&](int mt, int h) -> int { return 16 * (g >> 1) + 2 * (2 * mt + h) + (g & 1); };

  // weights of the (masked) scores: sums, and the V-scaled weights as P^T fragments
  uint32_t pb[4][2];
  auto softmax = [&](bool masked, const uint4& sc, bool scaled) {
    if (refs == 0 && !masked) {
      // the warp's first key (lane g = 0) gives the references
      nm[0] = -p.scale_log2 * __shfl_sync(kAll, s[0][0], t);
      nm[1] = -p.scale_log2 * __shfl_sync(kAll, s[0][1], t);
      refs = 2;
    }
    float xm = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[mt][e] = fmaf(s[mt][e], p.scale_log2, nm[e & 1]);
        xm = fmaxf(xm, s[mt][e]);
      }
    if (refs != 2 || __any_sync(kAll, xm > kHeadroom)) {
      // move the references to the largest score so far; with masked scores a
      // row may still have none (reference 0, no weights, nothing in O)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) mx = fmaxf(mx, fmaxf(s[mt][e], s[mt][e + 2]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, off));
        float sum = l[e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(kAll, sum, off);
        const bool fresh = sum == 0.f;                               // no weights yet
        const float shift = mx == -INFINITY ? 0.f : (fresh ? mx : fmaxf(mx, 0.f));
        const float alpha = fresh ? 1.f : ex2(-shift);
        nm[e] -= shift;
        l[e] *= alpha;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          s[mt][e] -= shift;
          s[mt][e + 2] -= shift;
        }
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[c][i][e] *= alpha;
            o[c][i][e + 2] *= alpha;
          }
      }
      // every row has a reference once the warp has seen an unmasked span;
      // until then the next span takes this path again
      if (refs != 2) refs = masked ? 1 : 2;
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
      float w[4], sv[2] = {1.f, 1.f};
      if (scaled) {
#pragma unroll
        for (int h = 0; h < 2; ++h) sv[h] = kv4::scale_of((word(sc, mt) >> (16 * h + 8 * (g & 1))) & 255u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = ex2(s[mt][e]);
        l[e & 1] += w[e];
      }
      pb[mt][0] = transpose8x8(pack_bf16(w[0] * sv[0], w[1] * sv[0]));
      pb[mt][1] = transpose8x8(pack_bf16(w[2] * sv[1], w[3] * sv[1]));
    }
  };
  auto pv = [&](const uint4 (&r)[8], int c) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const uint32_t we = word(r[i], mt >> 1), wo = word(r[i], 2 + (mt >> 1));   // even and odd channel
        const int e = 2 * (mt & 1);
        const uint32_t a0 = fma_bf16x2(pair(we, e), kOne, kMinus136), a1 = fma_bf16x2(pair(wo, e), kOne, kMinus136);
        const uint32_t a2 = fma_bf16x2(pair(we, e + 1), kOne, kMinus136), a3 = fma_bf16x2(pair(wo, e + 1), kOne, kMinus136);
        mma(o[c][i], a0, a1, a2, a3, pb[mt][0], pb[mt][1]);
      }
  };
  auto clear_s = [&]() {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[mt][e] = 0.f;
  };

  // ---------------------------------------------------------------- the warp's prefix spans
  int sp = warp;
  int id_k = page_of(sp, g >> 1), id_v = page_of(sp, t);           // this span's ids, then the next one's
  Blocks cur = blocks(id_k, id_v);
  if (sp < nsp) {
    load_k(buf[0], ksc[0], cur, 0);
    if (CPT > 1)
      load_k(buf[1], ksc[1], cur, 1);
    else
      load_v(buf[1], cur, 0);
    vsc = ldg16(v4 + cur.k * VB + 8 * D);
  }
  id_k = page_of(sp + kWarps, g >> 1);
  id_v = page_of(sp + kWarps, t);
  for (; sp < nsp; sp += kWarps) {
    const Blocks nxt = blocks(id_k, id_v);
    const bool more = sp + kWarps < nsp;
    id_k = page_of(sp + 2 * kWarps, g >> 1);
    id_v = page_of(sp + 2 * kWarps, t);
    clear_s();
    if (more) {
      // the next span's lines into L2 (159 -> 156 us on the batch above)
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        prefetch_l2(k4 + nxt.k * KB + c * 1024 + (4 * (g & 1) + t) * 128);
        prefetch_l2(v4 + nxt.v * VB + c * 1024 + g * 128);
      }
      prefetch_l2(k4 + nxt.k * KB + 8 * D);
      prefetch_l2(v4 + nxt.v * VB + 8 * D);
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      qk(buf[c & 1], ksc[c & 1], c);
      // piece c + 2 into the buffer just used
      if (c + 2 < CPT)
        load_k(buf[c & 1], ksc[c & 1], cur, c + 2);
      else if (c + 2 < 2 * CPT)
        load_v(buf[c & 1], cur, c + 2 - CPT);
      else if (more)
        load_k(buf[c & 1], ksc[c & 1], nxt, c + 2 - 2 * CPT);
    }
    bool masked = false;
    const int64_t v0 = k_begin + (int64_t)sp * kSpan;
    if (v0 + kSpan > k_end) {
      masked = true;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (v0 + key_of(mt, h) >= k_end) s[mt][2 * h] = s[mt][2 * h + 1] = -INFINITY;
    }
    if (WIN) {
      const int64_t p0 = km.pos(v0);
      if (p0 < P + kMaxNodes - p.window) {
        masked = true;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 2 * t + e;
          const int64_t lo = first_pos + (r < live ? p.depth[o0 + r / p.G] : 0);
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t pos = p0 + key_of(mt, h);
              if (!(pos < p.sinks || pos >= lo)) s[mt][2 * h + e] = -INFINITY;
            }
        }
      }
    }
    softmax(masked, vsc, true);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      constexpr int kPieces = 2 * CPT;
      const int i = CPT + c;                                       // this piece's number
      pv(buf[i & 1], c);
      if (i + 2 < kPieces)
        load_v(buf[i & 1], cur, c + 2);
      else if (more) {
        const int j = i + 2 - kPieces;                             // piece j of the next span
        if (j < CPT)
          load_k(buf[i & 1], ksc[i & 1], nxt, j);
        else
          load_v(buf[i & 1], nxt, j - CPT);
      }
    }
    if (more) vsc = ldg16(v4 + nxt.k * VB + 8 * D);
    cur = nxt;
  }

  // ---------------------------------------------------------------- the tree
  // (at most 8 nodes: rows <= 8), as one span of bf16 rows in the same
  // layout: nodes sit in block 0, lanes g < 2 (K) and t = 0 (V)
  if (nsp < total && warp == nsp % kWarps) {
    clear_s();
    const __nv_bfloat16* kt = reinterpret_cast<const __nv_bfloat16*>(p.k_tree) + ((int64_t)g_head * p.R + o0) * D;
    const __nv_bfloat16* vt = reinterpret_cast<const __nv_bfloat16*>(p.v_tree) + ((int64_t)g_head * p.R + o0) * D;
#pragma unroll 1
    for (int c = 0; c < CPT; ++c) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        const int n0 = key_of(mt, 0), n1 = key_of(mt, 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ch = c * 128 + 32 * t + 8 * (j >> 1) + 4 * (j & 1);
          uint2 x = make_uint2(0, 0), y = make_uint2(0, 0);
          if (n0 < n) x = __ldg(reinterpret_cast<const uint2*>(kt + (int64_t)n0 * D + ch));
          if (n1 < n) y = __ldg(reinterpret_cast<const uint2*>(kt + (int64_t)n1 * D + ch));
          if (C::QREG) {
#pragma unroll
            for (int cc = 0; cc < CPT; ++cc)
              if (cc == c) qk_step(cc, j, mt, x.x, y.x, x.y, y.y);
          } else {
            qk_step(c, j, mt, x.x, y.x, x.y, y.y);
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e;
      const int node = r / p.G;
      const uint64_t anc = r < live ? p.anc[o0 + node] : 0ull;
      const int dep = WIN && r < live ? p.depth[o0 + node] : 0;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = key_of(mt, h);
          bool vis = key < n && ((anc >> key) & 1ull);
          if (WIN && vis) {
            const int kd = p.depth[o0 + key];
            vis = P + kd < p.sinks || dep - (int64_t)kd < p.window;
          }
          if (!vis) s[mt][2 * h + e] = -INFINITY;
        }
    }
    softmax(true, vsc, false);
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        float acc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          uint32_t a[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int node = 16 * t + 2 * (2 * mt + h);            // keys node, node + 1 of block t
            uint32_t x = 0, y = 0;                                 // channels 16 i + 2 g, + 1 of each
            const uint32_t* src = reinterpret_cast<const uint32_t*>(vt + (int64_t)node * D + c * 128 + 16 * i + 2 * g);
            if (node < n) x = __ldg(src);
            if (node + 1 < n) y = __ldg(src + D / 2);
            a[2 * h] = __byte_perm(x, y, 0x5410);
            a[2 * h + 1] = __byte_perm(x, y, 0x7632);
          }
          mma(acc, a[0], a[1], a[2], a[3], pb[mt][0], pb[mt][1]);
        }
        // (o's index must be known when compiling)
#pragma unroll
        for (int ii = 0; ii < 8; ++ii)
          if (ii == i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][ii][e] += acc[e];
          }
      }
  }

  // ---------------------------------------------------------------- the warps' results joined
  // lane (g, t): rows 2 t, 2 t + 1, channels 16 i + 2 g, + 1 of each chunk
  if (!C::QREG) __syncthreads();                                   // the queries' shared memory is free
  float* so = smem + warp * 8 * C::OUT_PITCH;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float sum = l[e];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(kAll, sum, off);
    const int r = 2 * t + e;
    if (g == 0) {
      s_m[warp][r] = sum == 0.f ? -INFINITY : -nm[e];    // (a NaN sum has to show)
      s_l[warp][r] = sum;
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float2*>(so + r * C::OUT_PITCH + c * 128 + 16 * i + 2 * g) =
            make_float2(o[c][i][e], o[c][i][e + 2]);
  }
  __syncthreads();
  const bool direct = p.out != nullptr && nch == 1;
  const int64_t slot0 = partial_slot(s_id, b, g_head, 0, 0, p.Hkv, p.row_tiles, p.tile_stride, p.splits);
  for (int r = warp; r < live; r += kWarps) {
    float M = -INFINITY, L = 0.f, wt[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      wt[w] = s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - M);
      L += wt[w] * s_l[w][r];
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t row = row_at(r);
    if (!direct && lane == 0) p.ml_part[slot0 + (int64_t)r * p.splits] = make_float2(M, L);
    for (int ch = lane * 4; ch < D; ch += 128) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(smem + (w * 8 + r) * C::OUT_PITCH + ch);
        const float f = wt[w] * inv;
        a.x = fmaf(f, x.x, a.x);
        a.y = fmaf(f, x.y, a.y);
        a.z = fmaf(f, x.z, a.z);
        a.w = fmaf(f, x.w, a.w);
      }
      if (!direct) {
        *reinterpret_cast<float4*>(p.o_part + (slot0 + (int64_t)r * p.splits) * D + ch) = a;
      } else if (p.out_bf16) {
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + row + ch) =
            make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
      } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + row + ch) = a;
      }
    }
  }
}

template <int D, bool WIN>
cudaError_t launch_t(const AttnParams& p, cudaStream_t st) {
  const cudaError_t e = ensure_max_dynamic_smem<tv_attn_kv4_rows_kernel<D, WIN>>(Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dep(tv_attn_kv4_rows_kernel<D, WIN>, dim3(1, p.Hkv * p.splits, p.B), dim3(32 * kWarps),
                    Cfg<D>::SMEM, st, p);
}

template <bool WIN>
cudaError_t launch_d(const AttnParams& p, cudaStream_t s) {
  if (p.d == 128) return launch_t<128, WIN>(p, s);
  if (p.d == 256) return launch_t<256, WIN>(p, s);
  return launch_t<512, WIN>(p, s);
}

}  // namespace

bool kv4_rows_supported(const tv_desc* d, int G) { return d->dtype == TV_BF16 && d->max_nodes * G <= kRows; }

int kv4_rows_ctas_per_sm(int d) { return d == 128 ? Cfg<128>::CTAS : Cfg<256>::CTAS; }

int kv4_rows_key_tile() { return kSpan; }

cudaError_t launch_attn_kv4_rows(const AttnParams& p, cudaStream_t s) {
  return p.window > 0 ? launch_d<true>(p, s) : launch_d<false>(p, s);
}

}  // namespace tv
