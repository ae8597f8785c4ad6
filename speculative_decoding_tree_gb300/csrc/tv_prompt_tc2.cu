// Causal prompt attention on tcgen05 CTA pairs, bf16, head_dim 256 and 512.
//
// A pair takes 2 x 128 query rows (token, group head) of one sequence and KV
// head, 128 in each CTA, and 256 columns of V (head_dim 512: one of its two
// halves; the scores are then computed for each half, 3 products instead of 2,
// because an accumulator of 512 columns would leave tensor memory no room for
// scores).  M = 256 instructions (cta_group::2): each CTA holds its rows, half
// the keys of a K tile and half the columns of a V tile, so a K/V byte crosses
// from L2 once for 256 rows and a tile takes half the shared memory.
//   S(t) = Q K(t)^T goes to one of two 128-column buffers, the weights P(t)
//   over it as bf16, O += P(t) V(t).  S(t + 1) is issued before O += P(t) V(t).
//   A tile's softmax takes about 1250 clocks (a thread a row) and 750 more
//   from its last weights to the next scores where each waits for the other,
//   its products 2048 at head_dim 256: two warpgroups therefore take the tiles
//   in turn.  They share a row's reference (the exponent's offset): the group
//   of tile t hands it on as soon as it knows the tile's maximum, and rescales
//   O when that lies more than 2^8 above; each keeps its own sum.
//   200 rows x 16 heads behind 32768 keys, head_dim 256: 88 us (102 with the
//   products issued by a warp of one lane, 106 with one warpgroup).
//
//   warps 0-3, 4-7  softmax of the even and the odd tiles, epilogue
//   warp 8          TMA producer: Q, then K(0), K(1), V(0), K(2), V(1), ...;
//                   completion counts on the leader's barriers
//   warp 9          owns tensor memory; in the leader one lane's instructions
//                   are the products, every commit is multicast to both CTAs
// Every wait is bounded; the pair meets before tensor memory is freed.
#include <cuda.h>

#include "tc_ptx.cuh"
#include "tv_f32x2.cuh"
#include "tv_prompt.cuh"
#include "tv_tensormap.cuh"

namespace tv {
namespace {

using namespace tc;

constexpr int BM = 128;                         // query rows per CTA
constexpr int BN = kPromptTile;                 // keys of a tile
constexpr int KH = BN / 2;                      // keys of a K tile per CTA
constexpr uint32_t kHeader = 3 * 1024, kUnitOfs = 512;
constexpr uint32_t kRefOfs = 1024;              // [128] floats: a row's reference
constexpr uint32_t kSumOfs = 1536;              // [2][128] floats: the groups' sums
static_assert(kSumOfs + 1024 <= kHeader, "header");
constexpr int kThreads = 320;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescaleThreshold = 8.0f;       // rescale O when the maximum grows by more than 2^8

template <int D>
struct Cfg {
  static constexpr int DV = 256;                // value columns of a unit
  static constexpr int KC = 256;                // channels of a K slot
  static constexpr int KS = D / KC;             // slots of a K tile
  static constexpr uint32_t SLOT = KH * KC * 2; // 64 keys x KC channels of K, or 128 keys x DV / 2 columns of V
  static constexpr int SB = 2;                  // buffers of S; O follows them in tensor memory
  static constexpr uint32_t T_O = SB * 128;
  static constexpr int AHEAD = SB - 1;          // tiles S runs ahead
  static constexpr uint32_t Q_BYTES = BM * D * 2;
  static constexpr int NS = (232448 - kHeader - Q_BYTES) / SLOT;
  static constexpr uint32_t SMEM = kHeader + Q_BYTES + NS * SLOT;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_Q = 2 * NS, B_S = B_Q + 1, B_P = B_S + SB, B_O = B_P + 2 * SB,
                       B_REF = B_O + 2, B_SUM = B_REF + 8, B_TAIL = B_SUM + 4, B_FIN = B_TAIL + 1, NBARS = B_FIN + 1;
  static_assert(SMEM <= 232448, "shared memory over the 227 KB per-block limit");
  static_assert(NBARS * 8 + 16 <= kUnitOfs && T_O + DV <= 512, "header, tensor memory");
};

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
prompt_tc2_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                  const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_vr) {
  using C = Cfg<D>;
  constexpr int NS = C::NS, KS = C::KS, KC = C::KC, DV = C::DV, SB = C::SB;
  constexpr uint32_t SLOT = C::SLOT, T_O = C::T_O;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  PromptUnit& s_unit = *reinterpret_cast<PromptUnit*>(smem_raw + kUnitOfs);
  float* s_ref = reinterpret_cast<float*>(smem_raw + kRefOfs);
  float* s_sum = reinterpret_cast<float*>(smem_raw + kSumOfs);
  uint8_t* sQ = smem_raw + kHeader;
  uint8_t* ring = sQ + C::Q_BYTES;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto FULL = [&](int i) { return bar(C::B_FULL + i); };                  // used in the leader
  auto EMPTY = [&](int i) { return bar(C::B_EMPTY + i); };
  auto S_FULL = [&](int i) { return bar(C::B_S + i); };
  auto P_FULL = [&](int i, int h) { return bar(C::B_P + 2 * i + h); };    // used in the leader
  auto O_DONE = [&](int i) { return bar(C::B_O + i); };
  auto REF = [&](int q, int i) { return bar(C::B_REF + 2 * q + i); };    // row quarter q, tile parity i
  auto SUM = [&](int q) { return bar(C::B_SUM + q); };
  const uint32_t Q_FULL = bar(C::B_Q), TAIL = bar(C::B_TAIL), FIN = bar(C::B_FIN);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem_raw) & 1023u) {                 // the same in both CTAs of the pair
    dep_wait();
    if (tid == 0) set_status(p.status, TV_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(FULL(i), 2);                        // the leader's expect_tx arrive and the peer's arrive
      mbar_init(EMPTY(i), 1);
    }
    mbar_init(Q_FULL, 2);
    for (int i = 0; i < SB; ++i) {
      mbar_init(S_FULL(i), 1);
      mbar_init(P_FULL(i, 0), 8);                   // a tile's softmax warps of both CTAs
      mbar_init(P_FULL(i, 1), 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(O_DONE(i), 1);
      for (int q = 0; q < 4; ++q) mbar_init(REF(q, i), 1);
    }
    for (int q = 0; q < 4; ++q) mbar_init(SUM(q), 2);   // the quarter's two warps
    mbar_init(TAIL, 1);
    mbar_init(FIN, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (p.rows_per_tile < BM) {
    // pad rows of the query tile (G does not divide 128) hold zeros; the Q loads never write them
    const int pad = BM - p.rows_per_tile;
    for (int e = tid; e < (D / 64) * pad * 8; e += kThreads) {
      const int box = e / (pad * 8), r = p.rows_per_tile + (e / 8) % pad, c = e % 8;
      *reinterpret_cast<uint4*>(sQ + box * (BM * 128) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_vr);
  }
  dep_wait();
  dep_launch();
  const uint32_t rank = cluster_ctarank();          // 0 = leader
  int rest = (int)(blockIdx.x >> 1);
  const int s = rest % p.splits;
  rest /= p.splits;
  const int vh = rest % (D / DV);                   // which 256 columns of V
  rest /= D / DV;
  const int g = rest % p.Hkv;
  if (warp == 0) find_unit(p, rest / p.Hkv, &s_unit);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                               // both CTAs' barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the pair's rows and tiles (the same in every thread of both CTAs)
  const int b = s_unit.b, G = p.G, o0 = s_unit.o0, n = s_unit.n;
  const int64_t P = s_unit.P;
  const int tile_tokens = p.unit_tokens >> 1;
  const int pair0 = s_unit.i * p.unit_tokens, tok0 = pair0 + (int)rank * tile_tokens;   // first token of the pair, of the CTA
  const int Pt = (int)((P + BN - 1) / BN);
  const int t_begin = s * p.chunk_tiles;
  const int all = pair0 < n ? Pt + (min(n, pair0 + p.unit_tokens) - 1) / BN + 1 : 0;
  const int T = max(0, min(all - t_begin, p.chunk_tiles));

  if (T == 0) {
    // nothing for this pair
  } else if (warp == 8) {
    // ============================================================ producer
    const bool leader = rank == 0, rows_here = tok0 < n;
    if (lane == 0) {
      const uint32_t qf = map_to_cta(Q_FULL, 0);
      const uint32_t bytes = (uint32_t)p.rows_per_tile * 128u * (D / 64);
      if (leader) mbar_expect_tx(Q_FULL, bytes * (1 + (pair0 + tile_tokens < n)));
      if (rows_here)
        for (int kb = 0; kb < D / 64; ++kb)
          tma2_load_3d(smem_u32(sQ + kb * (BM * 128)), &tm_q, qf, kb * 64, g * G, o0 + tok0);
      if (!leader) mbar_arrive_cluster_relaxed(qf);
    }
    const int oob_row = p.paged ? (int)(p.num_pages * p.Hkv * kPageSize) : 0;
    auto page_pos = [&](int t) -> int64_t {         // first position of this lane's page of tile t, or -1 (none)
      const int tt = t_begin + t;
      if (!p.paged || t >= T || tt >= Pt || lane >= BN / kPageSize) return -1;
      const int64_t pos = (int64_t)tt * BN + lane * kPageSize;
      return pos < P ? pos : -1;
    };
    auto page_id = [&](int t) -> int {              // what the table holds (any number)
      const int64_t pos = page_pos(t);
      return pos < 0 ? 0 : p.page_table[(int64_t)b * p.max_pages + pos / kPageSize];
    };
    auto page_row = [&](int t, int pid) -> int {    // TMA row of a page id, checked where it is used
      if (page_pos(t) < 0) return -1;
      if (pid >= 0 && pid < p.num_pages) return (int)(((int64_t)pid * p.Hkv + g) * kPageSize);
      set_status(p.status, TV_DEV_BAD_PAGE);
      return oob_row;                               // out of range: the copy reads zeros
    };
    auto pages_in = [&](int64_t a, int len) -> int {   // pages of [a, a + len) with positions below P
      const int64_t e = min(a + len, P);
      return e > a ? (int)((e - a + kPageSize - 1) / kPageSize) : 0;
    };
    int pid_a = page_id(0), pid_b = page_id(1);
    int row_at[C::AHEAD + 1];                       // TMA rows of the tiles t, t - 1, ...
#pragma unroll
    for (int i = 0; i <= C::AHEAD; ++i) row_at[i] = -1;
    int j = 0, tail_uses = 0;
    bool ok = true;
    for (int t = 0; t < T + C::AHEAD && ok; ++t) {
#pragma unroll
      for (int i = C::AHEAD; i > 0; --i) row_at[i] = row_at[i - 1];
      row_at[0] = page_row(t, pid_a);
      pid_a = pid_b;
      pid_b = page_id(t + 2);
      for (int part = 0; part <= KS && ok; ++part) {   // the K slots of tile t, then V of tile t - AHEAD
        const bool isv = part == KS;
        const int tile = isv ? t - C::AHEAD : t;
        if (tile < 0 || tile >= T) continue;
        const int tt = t_begin + tile;
        const bool own = tt >= Pt;
        const int64_t first = own ? (int64_t)(tt - Pt) * BN : (int64_t)tt * BN;
        const int valid = (int)min((int64_t)BN, (own ? (int64_t)n : P) - first);   // keys of the tile that exist
        const bool fix = isv && valid < BN;         // V rows past the end become zeros: their weights are
        const int slot = j % NS, use = j / NS;
        if (use > 0 && !__all_sync(kAll, mbar_wait(EMPTY(slot), (use - 1) & 1, abort_flag, kWaitNs))) {
          ok = false;
          break;
        }
        uint8_t* dst = ring + slot * SLOT;
        const uint32_t full_l = map_to_cta(FULL(slot), 0);
        const uint32_t fb = fix ? map_to_cta(TAIL, rank) : full_l;
        uint32_t total = 2 * SLOT;                  // bytes both CTAs bring (the leader expects them all)
        if (p.paged && !own)
          total = (isv ? 2u * (uint32_t)pages_in(first, BN) * (DV / 128)
                       : (uint32_t)(pages_in(first, KH) + pages_in(first + KH, KH)) * (KC / 64)) *
                  (kPageSize * 128u);
        if (lane == 0) {
          if (fix) mbar_expect_tx(TAIL, total / 2);
          else if (leader) mbar_expect_tx(FULL(slot), total);
        }
        __syncwarp();
        if (own || !p.paged) {
          if (lane == 0) {
            const int64_t row =
                (own ? (int64_t)g * p.rows + o0 : ((int64_t)b * p.Hkv + g) * p.capacity) + first + (isv ? 0 : KH * rank);
            if (!isv) {                             // 64 keys x KC channels
              for (int bx = 0; bx < KC / 64; ++bx)
                tma2_load_2d(smem_u32(dst + bx * (KH * 128)), own ? &tm_kr : &tm_kc, fb, part * KC + bx * 64,
                             (int)row);
            } else {                                // 128 keys x DV / 2 columns
              for (int bx = 0; bx < DV / 128; ++bx)
                tma2_load_2d(smem_u32(dst + bx * (BN * 128)), own ? &tm_vr : &tm_vc, fb,
                             vh * DV + DV / 2 * (int)rank + bx * 64, (int)row);
            }
          }
        } else {
          const int my_row = isv ? row_at[C::AHEAD] : row_at[0];
          if (!isv) {
            const int pg = lane - 4 * (int)rank;    // lanes 4 rank .. 4 rank + 3 own the pages of this CTA's 64 keys
            if (pg >= 0 && pg < 4 && my_row >= 0)
              for (int bx = 0; bx < KC / 64; ++bx)
                tma2_load_2d(smem_u32(dst + bx * (KH * 128) + pg * kPageSize * 128), &tm_kc, fb, part * KC + bx * 64,
                             my_row);
          } else if (my_row >= 0) {
            for (int bx = 0; bx < DV / 128; ++bx)
              tma2_load_2d(smem_u32(dst + bx * (BN * 128) + lane * kPageSize * 128), &tm_vc, fb,
                           vh * DV + DV / 2 * (int)rank + bx * 64, my_row);
          }
        }
        __syncwarp();
        if (fix) {
          if (!__all_sync(kAll, mbar_wait_landed(TAIL, tail_uses & 1, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          ++tail_uses;
          const int nz = BN - valid;
          for (int e = lane; e < DV / 128 * nz * 8; e += 32) {
            const int bx = e / (nz * 8), r = valid + (e / 8) % nz, q16 = e % 8;
            *reinterpret_cast<uint4*>(dst + bx * (BN * 128) + r * 128 + q16 * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_release(full_l);   // the zeros must reach the pair's products
        } else if (!leader && lane == 0) {
          mbar_arrive_cluster_relaxed(full_l);      // the bytes themselves are counted by complete_tx
        }
        ++j;
      }
    }
    // drain: the copies of both CTAs (the leader's barriers count them) have landed before the pair's last barrier,
    // after a timeout too: a step that the leader no longer counts gets the time of a wait in the peer
    if (lane == 0 && !leader && !ok) wait_ns(kWaitNs);
    if (lane == 0 && leader) {
      int spare = 0;
      mbar_wait(Q_FULL, 0, &spare, kWaitNs);
      for (int jj = (j > NS ? j - NS : 0); jj < j; ++jj) mbar_wait(FULL(jj % NS), (jj / NS) & 1, &spare, kWaitNs);
    }
  } else if (warp == 9) {
    // ============================================================ MMA issuer (the leader's warp, one lane's instructions)
    if (rank == 0) {
      constexpr uint32_t ID_QK = idesc_bf16_f32(2 * BM, BN, 0, 0);
      constexpr uint32_t ID_PV = idesc_bf16_f32(2 * BM, DV, 0, 1);
      constexpr uint32_t HI = desc_hi(1024, 2);
      const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), k_lo = desc_lo(smem_u32(ring), 16),
                     v_lo = desc_lo(smem_u32(ring), BN * 128);
      const uint32_t tm = __shfl_sync(kAll, tmem, 0);
      const int nt = __shfl_sync(kAll, T, 0);
      const bool one = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(kAll, mbar_wait(bar, parity, abort_flag, kWaitNs)) != 0;
      };
      bool ok = wait(Q_FULL, 0);
      tc_fence_after();
      int slot = 0, phase = 0, sk = 0, sv = 0, pv = 0;   // ring; buffer of the next S, of the next P, the latter's phase
      auto next = [&] {
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      };
      for (int t = 0; t < nt + C::AHEAD && ok; ++t) {
        if (t < nt) {
          const uint32_t to = tm + (uint32_t)(sk * 128);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            ok = ok && wait(FULL(slot), phase);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = q_lo + ks * (KC / 64) * (BM * 128 / 16), bd = k_lo + slot * (SLOT / 16);
            if (one) {
              if (ks == 0) mma_pair_ss_lo<false>(to, a, bd, HI, ID_QK);
              else mma_pair_ss_lo<true>(to, a, bd, HI, ID_QK);
#pragma unroll
              for (int kk = 1; kk < KC / 16; ++kk)
                mma_pair_ss_lo<true>(to, a + (kk >> 2) * (BM * 128 / 16) + (kk & 3) * 2,
                                     bd + (kk >> 2) * (KH * 128 / 16) + (kk & 3) * 2, HI, ID_QK);
              mma_commit_pair(EMPTY(slot));
            }
            next();
          }
          if (!ok) break;
          if (one) mma_commit_pair(S_FULL(sk));
          sk = sk + 1 == SB ? 0 : sk + 1;
        }
        if (t >= C::AHEAD) {
          const int u = t - C::AHEAD;
          const uint32_t to = tm + T_O, pa = tm + (uint32_t)(sv * 128), bd = v_lo + slot * (SLOT / 16);
          ok = wait(FULL(slot), phase);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wait(P_FULL(sv, h), pv & 1);
            if (!ok) break;
            tc_fence_after();
            if (one) {
#pragma unroll
              for (int kq = 0; kq < BN / 32; ++kq) {
                const int kk = h * (BN / 32) + kq;
                if (kk == 0 && u == 0) mma_pair_ts_lo<false>(to, pa, bd, HI, ID_PV);
                else mma_pair_ts_lo<true>(to, pa + kk * 8, bd + kk * (16 * 128 / 16), HI, ID_PV);
              }
            }
          }
          if (!ok) break;
          if (one) {
            mma_commit_pair(EMPTY(slot));
            mma_commit_pair(O_DONE(u & 1));
          }
          next();
          if (++sv == SB) {
            sv = 0;
            ++pv;
          }
        }
      }
      if (one) mma_commit_pair(FIN);
      int spare = 0;                                // (not abort_flag: this wait also follows a timeout)
      mbar_wait(FIN, 0, &spare, kWaitNs);
      __syncwarp();
    }
  } else {
    // ============================================================ softmax and epilogue (own rows)
    const int grp = warp >> 2, quarter = warp & 3;  // this group's tiles: grp, grp + 2, ...
    const int r = quarter * 32 + lane;              // row of the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t obuf = tmem + lane_base + T_O;
    const float c2 = p.scale_log2;
    const int token = tok0 + r / G;                 // the row's place in its sequence
    const bool row_ok = r < p.rows_per_tile && token < n;
    const bool warp_live = __any_sync(kAll, row_ok);
    float m_ref = -INFINITY, l = 0.f;               // the row's reference as this group last saw it; its tiles' sum
    bool ok = true;
    for (int t = grp; t < T; t += 2) {
      const int sb = t % SB;
      if (!__all_sync(kAll, mbar_wait(S_FULL(sb), (t / SB) & 1, abort_flag, kWaitNs))) { ok = false; break; }
      tc_fence_after();
      const uint32_t sbuf = tmem + lane_base + (uint32_t)(sb * 128);
      if (warp_live) {
        uint32_t sv[BN];
        tmem_ld_x128(sbuf, sv);
        const int tt = t_begin + t;
        // the tile's keys 0 .. lim are seen by this row
        const int lim = row_ok ? (tt < Pt ? (int)min((int64_t)BN, P - (int64_t)tt * BN) - 1
                                          : min(BN, token + 1 - (tt - Pt) * BN) - 1)
                               : -1;
        if (__any_sync(kAll, lim < BN - 1)) {
#pragma unroll
          for (int e = 0; e < BN; ++e) sv[e] = e <= lim ? sv[e] : 0xff800000u;
        }
        float mq[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mq[q] = __uint_as_float(sv[q]);
#pragma unroll
        for (int e = 4; e < BN; e += 2)
          mq[(e >> 1) & 3] = fmax3(mq[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
        const float mx = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
        const float m_tile = mx == -INFINITY ? -INFINITY : mx * c2;
        float m_in = -INFINITY;                     // the reference after the tile before
        if (t > 0) {
          if (!__all_sync(kAll, mbar_wait(REF(quarter, (t - 1) & 1), ((t - 1) >> 1) & 1, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          m_in = s_ref[r];
        }
        const bool first = m_in == -INFINITY;
        const bool need = !first && m_tile > m_in + kRescaleThreshold;
        const float m_out = first || need ? fmaxf(m_in, m_tile) : m_in;
        if (__any_sync(kAll, need)) {
          // O holds the tiles before this one once the last of their products is done
          const int u = t - 1;
          if (!__all_sync(kAll, mbar_wait(O_DONE(u & 1), (u >> 1) & 1, abort_flag, kWaitNs))) { ok = false; break; }
          tc_fence_after();
          const float alpha = need ? ex2(m_in - m_out) : 1.f;
#pragma unroll 1
          for (int c = 0; c < DV; c += 16) {
            uint32_t rr[16];
            tmem_ld_x16(obuf + c, rr);
#pragma unroll
            for (int e = 0; e < 16; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st_x16(obuf + c, rr);
          }
        }
        s_ref[r] = m_out;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(REF(quarter, t & 1));
        if (m_out != m_ref) {                       // (from -inf: the sum is 0 and stays 0)
          l *= m_ref == -INFINITY ? 0.f : ex2(m_ref - m_out);
          m_ref = m_out;
        }
        const float nm = m_ref == -INFINITY ? 0.f : -m_ref;   // nothing seen yet: 2^-inf = 0
        const uint64_t c2x2 = pk2(c2, c2), nmx2 = pk2(nm, nm);
        uint64_t l4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int k = h * 64 + 2 * e;
            const float2 x = up2(ffma2(pk2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), c2x2, nmx2));
            const float2 y = make_float2(ex2(x.x), ex2(x.y));
            l4[e & 3] = fadd2(l4[e & 3], pk2(y.x, y.y));
            pk[e] = pack_bf16(y.x, y.y);
          }
          tmem_st_x32(sbuf + h * 32, pk);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_cta(P_FULL(sb, h), 0));
        }
        const float2 la = up2(fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3])));
        l += la.x + la.y;
      } else {
        // no row of this warp exists: whatever its lanes of P hold meets rows that are never read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(map_to_cta(P_FULL(sb, 0), 0));
          mbar_arrive_cluster(map_to_cta(P_FULL(sb, 1), 0));
        }
      }
    }
    // Epilogue: the groups' sums, brought to the row's last reference, are added; each group writes half of the columns,
    // through the query tile's shared memory, which no product reads any more: a thread stages 128 bytes of its row
    // (16-byte piece c at c ^ (row & 7)), then 8 lanes store them together.
    const int u = T - 1;
    // (the last products by their own barrier: the group that is done first may be two phases of O_DONE ahead)
    if (ok) ok = __all_sync(kAll, mbar_wait(FIN, 0, abort_flag, kWaitNs));
    if (ok && warp_live)
      ok = __all_sync(kAll, mbar_wait(REF(quarter, u & 1), (u >> 1) & 1, abort_flag, kWaitNs));
    if (ok && warp_live) {
      tc_fence_after();
      const float mf = s_ref[r];
      s_sum[grp * 128 + r] = m_ref == -INFINITY ? 0.f : l * ex2(m_ref - mf);
      __syncwarp();
      if (lane == 0) mbar_arrive(SUM(quarter));
      ok = __all_sync(kAll, mbar_wait(SUM(quarter), 0, abort_flag, kWaitNs));
      const float L = s_sum[r] + s_sum[128 + r];
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
      uint8_t* stage = sQ + warp * (32 * 128);
      const int my_s = (Pt + token / BN) / p.chunk_tiles;     // the row's last split
      const bool part = my_s > 0, write = ok && row_ok && s <= my_s;
      const int64_t slot = part ? prompt_slot(o0 + token, g * G + r % G, s, p.Hq, p.splits)
                                : (int64_t)(o0 + token) * p.Hq + g * G + r % G;
      // rows of each form in the warp: bf16 results, fp32 results, fp32 partials
      const unsigned parts = __ballot_sync(kAll, write && part), rows = __ballot_sync(kAll, write && !part);
      auto flush = [&](unsigned which, char* base, int64_t row_bytes, int64_t ofs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3), c = lane & 7;
          const int64_t at = __shfl_sync(kAll, slot, rr);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
          if (which >> rr & 1u) *reinterpret_cast<uint4*>(base + at * row_bytes + ofs + c * 16) = v;
        }
      };
      const int col0 = grp * (DV / 2);              // of the unit's columns
      if (rows && p.out_bf16) {
#pragma unroll 1
        for (int c = 0; c < DV / 2; c += 64) {
          __syncwarp();
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t rr[32];
            tmem_ld_x32(obuf + col0 + c + 32 * hf, rr);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q)
                w[q] = pack_bf16(__uint_as_float(rr[8 * e + 2 * q]) * inv, __uint_as_float(rr[8 * e + 2 * q + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * hf + e) ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
          flush(rows, reinterpret_cast<char*>(p.out), D * 2, (vh * DV + col0 + c) * 2);
        }
      }
      const unsigned wide = parts | (p.out_bf16 ? 0u : rows);
      if (wide) {
#pragma unroll 1
        for (int c = 0; c < DV / 2; c += 32) {
          uint32_t rr[32];
          tmem_ld_x32(obuf + col0 + c, rr);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_float4(__uint_as_float(rr[4 * e]) * inv, __uint_as_float(rr[4 * e + 1]) * inv,
                            __uint_as_float(rr[4 * e + 2]) * inv, __uint_as_float(rr[4 * e + 3]) * inv);
          __syncwarp();
          const int64_t ofs = (vh * DV + col0 + c) * 4;
          if (parts) flush(parts, reinterpret_cast<char*>(p.o_part), D * 4, ofs);
          if (wide & ~parts) flush(wide & ~parts, reinterpret_cast<char*>(p.out), D * 4, ofs);
        }
      }
      if (write && part && vh == 0 && grp == 0) p.ml_part[slot] = make_float2(mf, L);
    }
  }

  // ---------------------------------------------------------------- teardown (pair)
  // The leader's last commit (FIN) reaches both CTAs after every earlier one:
  // once the peer has seen it, no arrive of the pair's products is under way
  // to its shared memory, and the cluster barrier keeps either CTA from
  // leaving before the other is done.
  if (T > 0 && warp == 9 && lane == 0 && rank != 0) {
    int spare = 0;
    mbar_wait(FIN, 0, &spare, kWaitNs);
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(p.status, TV_DEV_TIMEOUT);
  cluster_sync_relaxed();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int D>
cudaError_t launch_d(const PromptParams& p, int64_t units, cudaStream_t st) {
  constexpr int DV = Cfg<D>::DV;
  CUtensorMap mq, mkc, mvc, mkr, mvr;
  const cuuint64_t row_bytes = (cuuint64_t)D * 2;
  {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.rows};
    cuuint64_t strides[2] = {row_bytes, row_bytes * p.Hq};
    cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(BM / p.G)};
    if (!encode_rows(&mq, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const cuuint64_t strides[1] = {row_bytes};
  {
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)p.Hkv * p.rows};
    cuuint32_t kbox[2] = {64, KH}, vbox[2] = {64, BN};
    if (!encode_rows(&mkr, p.k_rows, 2, dims, strides, kbox) || !encode_rows(&mvr, p.v_rows, 2, dims, strides, vbox))
      return cudaErrorInvalidValue;
  }
  mkc = mkr;                                        // no prefix: never read
  mvc = mvr;
  if (p.max_prefix > 0) {
    cuuint64_t dims[2] = {(cuuint64_t)D, p.paged ? (cuuint64_t)p.num_pages * p.Hkv * kPageSize
                                                 : (cuuint64_t)p.B * p.Hkv * p.capacity};
    cuuint32_t kbox[2] = {64, (cuuint32_t)(p.paged ? kPageSize : KH)};
    cuuint32_t vbox[2] = {64, (cuuint32_t)(p.paged ? kPageSize : BN)};
    if (!encode_rows(&mkc, p.k_cache, 2, dims, strides, kbox) || !encode_rows(&mvc, p.v_cache, 2, dims, strides, vbox))
      return cudaErrorInvalidValue;
  }
  const cudaError_t e = ensure_max_dynamic_smem<prompt_tc2_kernel<D>>((int)Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dep(prompt_tc2_kernel<D>, dim3((unsigned)(units * p.Hkv * (D / DV) * p.splits * 2)), dim3(kThreads),
                    Cfg<D>::SMEM, st, p, mq, mkc, mvc, mkr, mvr);
}

}  // namespace

cudaError_t launch_prompt_tc2(const PromptParams& p, int64_t units, cudaStream_t st) {
  return p.d == 256 ? launch_d<256>(p, units, st) : launch_d<512>(p, units, st);
}

}  // namespace tv
