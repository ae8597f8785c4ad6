// Causal prompt attention on tcgen05 with fp32 accuracy: fp32 inputs, and bf16
// ones whose head groups the other kernels' tiles do not take.
//
// An fp32 number is the sum of three bf16 numbers, x = x1 + x2 + x3 with
// |x2| <= 2^-8 |x1| and |x3| <= 2^-16 |x1| (8 bits each, remainders exact), and
// a product of two such sums is, to about 2^-24 of it,
//     x1 y1 + (x1 y2 + x2 y1 + x2 y2 + x1 y3 + x3 y1),
// six bf16 products whose terms are exact in fp32.  The tensor cores' adder
// drops low bits of its accumulator at every step, so the large products and
// the small ones have accumulators of their own for S = Q K^T, and the tile's
// P V (small products first, 8 steps of large ones after) is added to O in
// registers, rounded to nearest.  Six products at 4096 multiply-adds a clock
// are 5 times the rate of the fp32 units.
//
// Two kernels.  The first splits every number once, resolving pages, ends and
// the grouping of heads, into blocks of 128 rows x 64 channels x 3 parts that
// lie in memory as the matrix unit reads them (rows of 128 bytes, 16-byte
// piece c at c ^ (row & 7)); rows that do not exist are zeros.  (Splitting in
// the attention kernel itself, for every unit again, took 158 - 208 us for
// 2000 rows x 4 heads at head_dim 256 where this took 108, and takes 84 - 89
// now.)  The second copies those blocks to shared memory,
// 48 KB each, and multiplies.
//
// A unit is 128 query rows (token, group head) of one sequence and KV head and
// 128 columns of V (the scores are computed for each block of columns: 1.5
// times the products at head_dim 256, which the small calls of this type pay
// for with twice the CTAs).
//
//   warps 0-7  softmax: two threads a row, each with 64 keys of a tile's
//              scores and 64 columns of O; the pair exchanges its maxima
//   warp 8     lane 0 copies: per key tile Q and K of each 64 channels (Q's
//              parts do not all fit), then two blocks of V
//   warp 9     owns tensor memory; one lane's instructions are the products
// Every wait is bounded.
#include <cuda.h>

#include "tc_ptx.cuh"
#include "tv_prompt.cuh"

namespace tv {
namespace {

using namespace tc;

constexpr int BM = 128;                         // query rows of a unit
constexpr int BN = kPromptTile;                 // keys of a tile
constexpr int DV = 128;                         // columns of V of a unit
constexpr int CH = 64;                          // channels of a slot
constexpr uint32_t PART = 128 * CH * 2;         // bytes of one bf16 part of a slot
constexpr uint32_t SLOT = 3 * PART;
constexpr int NS = 4;                           // (even: DV / CH = 2 slots of V lie side by side)
static_assert(DV / CH == 2 && NS % 2 == 0, "V's slots");
constexpr uint32_t kHeader = 3 * 1024;
constexpr uint32_t SMEM = kHeader + NS * SLOT;
static_assert(SMEM <= 232448, "shared memory over the 227 KB per-block limit");
constexpr int kThreads = 320;
constexpr int kSoftmaxWarps = 8;
constexpr uint64_t kWaitNs = 1000000000ull;

constexpr int B_FULL = 0, B_EMPTY = NS, B_S = 2 * NS, B_P = B_S + 1, B_OFULL = B_P + 1, B_OEMPTY = B_OFULL + 1,
              B_XCH = B_OEMPTY + 1, B_FIN = B_XCH + 8, NBARS = B_FIN + 1;
constexpr uint32_t kXchOfs = 512;               // [2 parity][2 half][128 rows] floats
constexpr uint32_t kUnitOfs = kXchOfs + 2048;
static_assert(kUnitOfs + sizeof(PromptUnit) <= kHeader && NBARS * 8 + 16 <= kXchOfs, "header");

// tensor memory: large products of S (then parts 1 and 2 of P), small products
// of S (then part 3 of P), P V of a tile
constexpr uint32_t T_BIG = 0, T_SMALL = 128, T_O = 256, T_COLS = 512;

// a pair as bf16, and what is left of it
__device__ __forceinline__ uint32_t part_of(float& a, float& b) {
  const uint32_t w = pack_bf16(a, b);
  a -= __uint_as_float(w << 16);
  b -= __uint_as_float(w & 0xffff0000u);
  return w;
}

// Blocks in the workspace, each SLOT bytes: K of every (KV head, key tile,
// 64 channels), then V, then Q of every (KV head, unit, 64 channels).  Key
// tiles: ptiles of each sequence's prefix, then the rows' own, which start at
// row / 128 + b for the sequence b that starts at `row` (ranges never meet: a
// sequence of n rows takes ceil(n / 128) of the n / 128 + 1 or more before the
// next); units likewise, counted in query rows.
struct Blocks {
  int ptiles;                                       // of max_prefix
  int64_t ktiles, qtiles;                           // per KV head
  __host__ __device__ Blocks(int64_t max_prefix, int64_t rows, int B, int G) {
    ptiles = (int)((max_prefix + BN - 1) / BN);
    ktiles = (int64_t)B * ptiles + rows / BN + B;
    qtiles = rows * G / BM + B;
  }
  __host__ __device__ int64_t own(int b, int64_t row, int B) const { return (int64_t)B * ptiles + row / BN + b; }
  __host__ __device__ int64_t unit(int b, int64_t row, int G) const { return row * G / BM + b; }
  // block of chunk c of head g's tile; kind 0 K, 1 V, 2 Q
  __host__ __device__ int64_t at(int kind, int Hkv, int chunks, int g, int64_t tile, int c) const {
    const int64_t per = kind == 2 ? qtiles : ktiles;
    return (kind * Hkv * ktiles + g * per + tile) * chunks + c;
  }
};

// The last sequence whose first tile (of `start`) is at or before `tile`.
template <typename F>
__device__ __forceinline__ int sequence_of(int B, int64_t tile, F start) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A CTA splits one tile's 64 channels: K and V of a key tile, or Q of a unit.
template <bool BF16, int D>
__global__ void __launch_bounds__(256) prompt_split_kernel(const __grid_constant__ PromptParams p) {
  constexpr int KC = D / CH;
  __shared__ int64_t s_at[128];                     // first element of a row, -1: none (zeros)
  __shared__ int s_any;
  const int tid = threadIdx.x;
  dep_wait();
  dep_launch();
  const Blocks blocks(p.max_prefix, p.rows, p.B, p.G);
  const int g = blockIdx.y / KC, c = blockIdx.y % KC;
  const int64_t x = blockIdx.x, prefix_tiles = (int64_t)p.B * blocks.ptiles;
  const bool isq = x >= blocks.ktiles, own = !isq && x >= prefix_tiles;
  const int64_t tile = isq ? x - blocks.ktiles : x;
  int64_t o0, n, first = 0, at = -1;                // the tile's first row of its kind
  int b = 0;
  if (isq || own) {
    b = isq ? sequence_of(p.B, tile, [&](int i) { return blocks.unit(i, p.row_offsets[i], p.G); })
            : sequence_of(p.B, tile, [&](int i) { return blocks.own(i, p.row_offsets[i], p.B); });
  } else {
    b = (int)(tile / blocks.ptiles);
    first = (tile - (int64_t)b * blocks.ptiles) * BN;
  }
  if (tid == 0) s_any = 0;
  __syncthreads();
  if (prompt_rows(p.row_offsets, b, p.rows, p.max_rows, p.status, &o0, &n) && n > 0 && tid < 128) {
    if (isq) {
      const int64_t m = (tile - blocks.unit(b, o0, p.G)) * BM + tid;
      if (m >= 0 && m < n * p.G) at = ((o0 + m / p.G) * p.Hq + g * p.G + m % p.G) * D;
    } else if (own) {
      const int64_t i = (tile - blocks.own(b, o0, p.B)) * BN + tid;
      if (i >= 0 && i < n) at = ((int64_t)g * p.rows + o0 + i) * D;
    } else {
      const int64_t P = clamp_prefix(p.prefix_len[b], p.max_prefix, p.capacity), key = first + tid;
      if (key < P && !p.paged) {
        at = (((int64_t)b * p.Hkv + g) * p.capacity + key) * D;
      } else if (key < P) {
        const int pid = p.page_table[(int64_t)b * p.max_pages + key / kPageSize];
        if (pid >= 0 && pid < p.num_pages) at = (((int64_t)pid * p.Hkv + g) * kPageSize + key % kPageSize) * D;
        else set_status(p.status, TV_DEV_BAD_PAGE);  // reads as zeros
        s_any = 1;
      }
    }
    if (at >= 0) s_any = 1;
  }
  if (tid < 128) s_at[tid] = at;
  __syncthreads();
  if (!s_any) return;                               // no unit reads this tile
  const int col = 4 * (tid & 15);
  for (int kind = isq ? 2 : 0; kind < (isq ? 3 : 2); ++kind) {
    const void* src = isq ? p.q : kind == 0 ? (own ? p.k_rows : p.k_cache) : (own ? p.v_rows : p.v_cache);
    uint8_t* base = reinterpret_cast<uint8_t*>(p.split) + blocks.at(kind, p.Hkv, KC, g, tile, c) * SLOT;
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t e = s_at[16 * i + (tid >> 4)];
      v[i] = make_float4(0, 0, 0, 0);
      if (e >= 0) {
        if (BF16) {
          const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(src) + e + c * CH + col);
          v[i] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                             __uint_as_float(w.y & 0xffff0000u));
        } else {
          v[i] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(src) + e + c * CH + col);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 16 * i + (tid >> 4);
      uint8_t* dst = base + r * 128 + ((((tid & 15) >> 1) ^ (r & 7)) << 4) + ((tid & 1) << 3);
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        uint2 w;
        w.x = part_of(v[i].x, v[i].y);
        w.y = part_of(v[i].z, v[i].w);
        *reinterpret_cast<uint2*>(dst + part * PART) = w;
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_f32_kernel(const __grid_constant__ PromptParams p) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr int KC = D / CH;                    // channel slots of Q and of K
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  PromptUnit& s_unit = *reinterpret_cast<PromptUnit*>(smem_raw + kUnitOfs);
  float* xch = reinterpret_cast<float*>(smem_raw + kXchOfs);
  uint8_t* ring = smem_raw + kHeader;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto FULL = [&](int i) { return bar(B_FULL + i); };
  auto EMPTY = [&](int i) { return bar(B_EMPTY + i); };
  auto XCH = [&](int q, int i) { return bar(B_XCH + 2 * q + i); };   // row quarter q, parity i
  const uint32_t S_FULL = bar(B_S), P_FULL = bar(B_P), O_FULL = bar(B_OFULL), O_EMPTY = bar(B_OEMPTY),
                 FIN = bar(B_FIN);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem_raw) & 1023u) {                 // the layout needs a 1 KB aligned window
    dep_wait();
    if (tid == 0) set_status(p.status, TV_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(FULL(i), 1);
      mbar_init(EMPTY(i), 1);
    }
    mbar_init(S_FULL, 1);
    mbar_init(P_FULL, kSoftmaxWarps);
    mbar_init(O_FULL, 1);
    mbar_init(O_EMPTY, kSoftmaxWarps);
    for (int q = 0; q < 4; ++q)
      for (int i = 0; i < 2; ++i) mbar_init(XCH(q, i), 2);   // the row quarter's two warps
    mbar_init(FIN, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), T_COLS);
    tmem_relinquish();
  }
  dep_wait();
  dep_launch();
  int rest = blockIdx.x;
  const int s = rest % p.splits;
  rest /= p.splits;
  const int vq = rest % (D / DV);                   // which 128 columns of V
  rest /= D / DV;
  const int g = rest % p.Hkv;
  if (warp == 0) find_unit(p, rest / p.Hkv, &s_unit);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the unit's rows and tiles (the same in every thread)
  const int b = s_unit.b, G = p.G;
  const int64_t o0 = s_unit.o0, n = s_unit.n, P = s_unit.P;
  const int64_t nrows = n * G;
  const int64_t m0 = (int64_t)s_unit.i * BM;
  const int64_t last = min(nrows, m0 + BM) - 1;
  const int Pt = (int)((P + BN - 1) / BN);
  const int t_begin = s * p.chunk_tiles;
  const int all = m0 < nrows ? Pt + (int)(last / G / BN) + 1 : 0;
  const int T = max(0, min(all - t_begin, p.chunk_tiles));

  if (T == 0) {
    // nothing for this CTA
  } else if (warp == 8) {
    // ============================================================ copies
    if (lane == 0) {
      const Blocks blocks(p.max_prefix, p.rows, p.B, G);
      const uint8_t* split = reinterpret_cast<const uint8_t*>(p.split);
      const int64_t unit = blocks.unit(b, o0, G) + s_unit.i;
      constexpr int PER = 2 * KC + DV / CH;         // slots of a tile
      int u = 0;
      bool ok = true;
      for (int t = 0; t < T && ok; ++t) {
        const int tt = t_begin + t;
        const int64_t tile = tt < Pt ? (int64_t)b * blocks.ptiles + tt : blocks.own(b, o0, p.B) + tt - Pt;
        for (int c = 0; c < PER; ++c, ++u) {
          const int slot = u % NS, use = u / NS;
          if (use > 0 && !mbar_wait(EMPTY(slot), (use - 1) & 1, abort_flag, kWaitNs)) { ok = false; break; }
          const int64_t block = c >= 2 * KC ? blocks.at(1, p.Hkv, KC, g, tile, vq * (DV / CH) + c - 2 * KC)
                                : c & 1     ? blocks.at(0, p.Hkv, KC, g, tile, c >> 1)
                                            : blocks.at(2, p.Hkv, KC, g, unit, c >> 1);
          mbar_expect_tx(FULL(slot), SLOT);
          bulk_load(smem_u32(ring + slot * SLOT), split + block * SLOT, SLOT, FULL(slot));
        }
      }
      // drain: every copy has landed before the CTA exits, after a timeout too
      int spare = 0;
      for (int j = (u > NS ? u - NS : 0); j < u; ++j) mbar_wait(FULL(j % NS), (j / NS) & 1, &spare, kWaitNs);
    }
  } else if (warp == 9) {
    // ============================================================ MMA issuer (the whole warp, one lane's instructions)
    constexpr uint32_t ID_QK = idesc_bf16_f32(BM, BN, 0, 0);
    constexpr uint32_t ID_PV = idesc_bf16_f32(BM, DV, 0, 1);
    constexpr uint32_t HI = desc_hi(1024, 2), P16 = PART / 16;
    const uint32_t ring_lo = desc_lo(smem_u32(ring), 16), v_lo = desc_lo(smem_u32(ring), SLOT);
    const uint32_t tm = __shfl_sync(kAll, tmem, 0);
    const int nt = __shfl_sync(kAll, T, 0);
    const bool one = elect_one();
    auto wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(kAll, mbar_wait(bar, parity, abort_flag, kWaitNs)) != 0;
    };
    int slot = 0, phase = 0;
    auto next = [&] {
      if (++slot == NS) {
        slot = 0;
        phase ^= 1;
      }
    };
    bool ok = true;
    for (int t = 0; t < nt && ok; ++t) {
      for (int c = 0; c < KC && ok; ++c) {
        const int qs = slot;
        ok = wait(FULL(qs), phase);
        if (!ok) break;
        next();
        const int ks = slot;
        ok = wait(FULL(ks), phase);
        if (!ok) break;
        next();
        tc_fence_after();
        const uint32_t q = ring_lo + qs * (SLOT / 16), k = ring_lo + ks * (SLOT / 16);
        if (one) {
          // parts a of Q and b of K, 16 channels a step
          auto product = [&](uint32_t a, uint32_t b, uint32_t to) {
#pragma unroll
            for (int kk = 0; kk < CH / 16; ++kk) mma_ss_lo<true>(tm + to, a + kk * 2, b + kk * 2, HI, ID_QK);
          };
          if (c == 0) {
            mma_ss_lo<false>(tm + T_SMALL, q, k + 2 * P16, HI, ID_QK);
            mma_ss_lo<false>(tm + T_BIG, q, k, HI, ID_QK);
          } else {
            mma_ss_lo<true>(tm + T_SMALL, q, k + 2 * P16, HI, ID_QK);
            mma_ss_lo<true>(tm + T_BIG, q, k, HI, ID_QK);
          }
#pragma unroll
          for (int kk = 1; kk < CH / 16; ++kk) {
            mma_ss_lo<true>(tm + T_SMALL, q + kk * 2, k + 2 * P16 + kk * 2, HI, ID_QK);
            mma_ss_lo<true>(tm + T_BIG, q + kk * 2, k + kk * 2, HI, ID_QK);
          }
          product(q + 2 * P16, k, T_SMALL);
          product(q + P16, k + P16, T_SMALL);
          product(q, k + P16, T_SMALL);
          product(q + P16, k, T_SMALL);
          mma_commit(EMPTY(qs));
          mma_commit(EMPTY(ks));
        }
      }
      if (!ok) break;
      if (one) mma_commit(S_FULL);
      ok = wait(P_FULL, t & 1) && (t == 0 || wait(O_EMPTY, (t - 1) & 1));
      if (!ok) break;
      // both blocks of V at once: 128 columns (64 run at 0.64 of the rate).  A tile's slots are even in number and so is
      // the ring, so the two are neighbours, a slot apart.
      const int vs = slot;
      ok = wait(FULL(vs), phase) && wait(FULL(vs + 1), phase);
      if (!ok) break;
      next();
      next();
      tc_fence_after();
      if (one) {
        const uint32_t b = v_lo + vs * (SLOT / 16), to = tm + T_O;
        auto product = [&](uint32_t pa, uint32_t part, bool rest) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            if (rest || kk > 0) mma_ts_lo<true>(to, tm + pa + kk * 8, part + kk * (16 * 128 / 16), HI, ID_PV);
        };
        mma_ts_lo<false>(to, tm + T_BIG, b + 2 * P16, HI, ID_PV);
        product(T_BIG, b + 2 * P16, false);
        product(T_SMALL, b, true);
        product(T_BIG + 64, b + P16, true);
        product(T_BIG, b + P16, true);
        product(T_BIG + 64, b, true);
        product(T_BIG, b, true);
        mma_commit(EMPTY(vs));
        mma_commit(EMPTY(vs + 1));
      }
      if (!ok) break;
      if (one) mma_commit(O_FULL);
    }
    // every product issued has finished before tensor memory is freed
    if (one) mma_commit(FIN);
    int spare = 0;                                  // (not abort_flag: this wait also follows a timeout)
    mbar_wait(FIN, 0, &spare, kWaitNs);
    __syncwarp();
  } else {
    // ============================================================ softmax and epilogue
    const int half = warp >> 2;                     // keys 64 half .. of a tile, columns 64 half .. of O
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;              // row of the unit == TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const float c2 = p.scale_log2;
    const int64_t m = m0 + r;
    const bool row_ok = m < nrows;
    const int token = row_ok ? (int)(m / G) : 0;    // the row's place in its sequence
    float m_run = -INFINITY, l = 0.f;
    float o[64];
#pragma unroll
    for (int e = 0; e < 64; ++e) o[e] = 0.f;
    int xt = 0;
    bool ok = true;
    // the row's two threads exchange one float
    auto exchange = [&](float mine, float& theirs) -> bool {
      float* xb = xch + (xt & 1) * 256;
      xb[half * 128 + r] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(XCH(quarter, xt & 1));
      const bool in = __all_sync(kAll, mbar_wait(XCH(quarter, xt & 1), (xt >> 1) & 1, abort_flag, kWaitNs));
      ++xt;
      theirs = xb[(half ^ 1) * 128 + r];
      return in;
    };
    for (int t = 0; t < T; ++t) {
      if (!__all_sync(kAll, mbar_wait(S_FULL, t & 1, abort_flag, kWaitNs))) { ok = false; break; }
      tc_fence_after();
      float sv[64];
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t big[16], small[16];
        tmem_ld_x16(lanes + T_BIG + half * 64 + c, big);
        tmem_ld_x16(lanes + T_SMALL + half * 64 + c, small);
#pragma unroll
        for (int e = 0; e < 16; ++e) sv[c + e] = __uint_as_float(big[e]) + __uint_as_float(small[e]);
      }
      tc_fence_before();                            // (the partner writes over these columns after the exchange)
      const int tt = t_begin + t;
      // this half's keys 0 .. lim are seen by the row
      const int lim = row_ok ? (tt < Pt ? (int)min((int64_t)BN, P - (int64_t)tt * BN) - 1
                                        : min(BN, token + 1 - (tt - Pt) * BN) - 1) - 64 * half
                             : -1;
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 64; ++e) {
        sv[e] = e <= lim ? sv[e] * c2 : -INFINITY;
        mx = fmaxf(mx, sv[e]);
      }
      float other;
      if (!exchange(mx, other)) { ok = false; break; }
      tc_fence_after();
      const float m_new = fmaxf(m_run, fmaxf(mx, other));
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2(m_run - ref);
      m_run = m_new;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t part[3][16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x = ex2(sv[c + 2 * e] - ref), y = ex2(sv[c + 2 * e + 1] - ref);
          sum[e & 3] += x + y;
          part[0][e] = part_of(x, y);
          part[1][e] = part_of(x, y);
          part[2][e] = pack_bf16(x, y);
        }
        const uint32_t at = half * 32 + c / 2;
        tmem_st_x16(lanes + T_BIG + at, part[0]);
        tmem_st_x16(lanes + T_BIG + 64 + at, part[1]);
        tmem_st_x16(lanes + T_SMALL + at, part[2]);
      }
      l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(P_FULL);
      if (!__all_sync(kAll, mbar_wait(O_FULL, t & 1, abort_flag, kWaitNs))) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t rr[16];
        tmem_ld_x16(lanes + T_O + half * 64 + c, rr);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[c + e] = fmaf(o[c + e], alpha, __uint_as_float(rr[e]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(O_EMPTY);
    }
    float l2 = 0.f;
    if (ok) ok = exchange(l, l2);
    if (ok && row_ok) {
      const float L = half == 0 ? l + l2 : l2 + l;
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
      const int my_s = (Pt + token / BN) / p.chunk_tiles;     // the row's last split
      if (s <= my_s) {
        const bool split = my_s > 0;
        const int h = g * G + (int)(m % G);
        const int64_t at = split ? prompt_slot(o0 + token, h, s, p.Hq, p.splits) : (o0 + token) * p.Hq + h;
        const int64_t to = at * D + vq * DV + half * 64;
        if (!split && p.out_bf16) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + to);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pack_bf16(o[8 * e + 2 * q] * inv, o[8 * e + 2 * q + 1] * inv);
            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>((split ? p.o_part : reinterpret_cast<float*>(p.out)) + to);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            dst[e] = make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
        }
        if (split && vq == 0 && half == 0) p.ml_part[at] = make_float2(m_run, L);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(p.status, TV_DEV_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, T_COLS);
  }
}

template <bool BF16, int D>
cudaError_t launch_d(const PromptParams& p, int64_t units, cudaStream_t st) {
  const Blocks blocks(p.max_prefix, p.rows, p.B, p.G);
  const dim3 grid((unsigned)(blocks.ktiles + blocks.qtiles), p.Hkv * (D / CH));
  cudaError_t e = launch_dep(prompt_split_kernel<BF16, D>, grid, dim3(256), 0, st, p);
  if (e != cudaSuccess) return e;
  e = ensure_max_dynamic_smem<prompt_f32_kernel<D>>((int)SMEM);
  if (e != cudaSuccess) return e;
  return launch_dep(prompt_f32_kernel<D>, dim3((unsigned)(units * p.Hkv * (D / DV) * p.splits)), dim3(kThreads), SMEM, st,
                    p);
}

}  // namespace

int64_t prompt_f32_bytes(const tv_desc* d, int64_t rows) {
  const Blocks blocks(d->max_prefix, rows, d->batch, d->num_q_heads / d->num_kv_heads);
  int64_t t;
  if (blocks.ktiles + blocks.qtiles > ((int64_t)1 << 31) - 1 || d->num_kv_heads * (d->head_dim / CH) > kMaxGridYZ ||
      __builtin_mul_overflow(2 * blocks.ktiles + blocks.qtiles, (int64_t)d->num_kv_heads * (d->head_dim / CH), &t) ||
      __builtin_mul_overflow(t, (int64_t)SLOT, &t))
    return -1;
  return t;
}

cudaError_t launch_prompt_f32(const PromptParams& p, int dtype, int64_t units, cudaStream_t s) {
  const bool bf = dtype == TV_BF16;
  if (p.d == 128) return bf ? launch_d<true, 128>(p, units, s) : launch_d<false, 128>(p, units, s);
  if (p.d == 256) return bf ? launch_d<true, 256>(p, units, s) : launch_d<false, 256>(p, units, s);
  return bf ? launch_d<true, 512>(p, units, s) : launch_d<false, 512>(p, units, s);
}

}  // namespace tv
