// Causal prompt attention on tcgen05 CTA pairs, bf16, head_dim 256 and 512.
//
// A pair takes 2 x 128 query rows (token, group head) of one sequence and KV
// head, 128 in each CTA, and 256 columns of V (head_dim 512: one of its two
// halves; the scores are then computed for each half, 3 products instead of 2,
// because an accumulator of 512 columns would leave tensor memory no room for
// scores).  M = 256 instructions (cta_group::2): each CTA holds its rows, half
// the keys of a K tile and half the columns of a V tile, so a K/V byte crosses
// from L2 once for 256 rows and a tile takes half the shared memory.
//   S(t) = Q K(t)^T in one of two 128-column buffers; the weights P(t) go over
//   them as bf16; O += P(t) V(t).  S(t + 1) is issued before O += P(t) V(t), so
//   the softmax of a tile has the time of the products of another: 2048 clocks
//   at head_dim 256, about twice what one warpgroup a CTA needs (a row a thread).
//
//   warps 0-3  softmax and epilogue of the CTA's rows
//   warp 4     TMA producer: Q, then K(0), K(1), V(0), K(2), V(1), ... in 32 KB
//              slots; completion counts on the leader's barriers
//   warp 5     owns tensor memory; the leader's lane 0 issues the products and
//              multicasts every commit to both CTAs
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
constexpr int DV = 256;                         // value columns per unit
constexpr uint32_t SLOT = 32768;                // 64 keys x 256 channels of K, or 128 keys x 128 columns of V
constexpr uint32_t kHeader = 3072, kUnitOfs = 1024;
constexpr int kThreads = 192;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescaleThreshold = 8.0f;       // rescale O when the maximum grows by more than 2^8

template <int D>
struct Cfg {
  static constexpr uint32_t Q_BYTES = BM * D * 2;
  static constexpr int NS = (232448 - kHeader - Q_BYTES) / SLOT;
  static constexpr int KS = D / 256;            // slots of a K tile
  static constexpr uint32_t SMEM = kHeader + Q_BYTES + NS * SLOT;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_Q = 2 * NS, B_S = B_Q + 1, B_P = B_S + 2, B_O = B_P + 4,
                       B_TAIL = B_O + 2, B_FIN = B_TAIL + 1, NBARS = B_FIN + 1;
  static_assert(SMEM <= 232448, "shared memory over the 227 KB per-block limit");
};

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
prompt_tc2_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                  const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_vr) {
  using C = Cfg<D>;
  constexpr int NS = C::NS, KS = C::KS;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + C::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  PromptUnit& s_unit = *reinterpret_cast<PromptUnit*>(smem_raw + kUnitOfs);
  uint8_t* sQ = smem_raw + kHeader;
  uint8_t* ring = sQ + C::Q_BYTES;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto FULL = [&](int i) { return bar(C::B_FULL + i); };                  // used in the leader
  auto EMPTY = [&](int i) { return bar(C::B_EMPTY + i); };
  auto S_FULL = [&](int i) { return bar(C::B_S + i); };
  auto P_FULL = [&](int i, int h) { return bar(C::B_P + 2 * i + h); };    // used in the leader
  auto O_DONE = [&](int i) { return bar(C::B_O + i); };
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(S_FULL(i), 1);
      mbar_init(P_FULL(i, 0), 8);                   // the softmax warps of both CTAs
      mbar_init(P_FULL(i, 1), 8);
      mbar_init(O_DONE(i), 1);
    }
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
  if (warp == 5) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 4 && lane == 0) {
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
  } else if (warp == 4) {
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
    int pid_a = page_id(0), pid_b = page_id(1), row_k = -1, row_v = -1;
    int j = 0, tail_uses = 0;
    bool ok = true;
    for (int t = 0; t <= T && ok; ++t) {
      row_v = row_k;
      row_k = page_row(t, pid_a);
      pid_a = pid_b;
      pid_b = page_id(t + 2);
      for (int part = 0; part <= KS && ok; ++part) {   // the K slots of tile t, then V of tile t - 1
        const bool isv = part == KS;
        const int tile = isv ? t - 1 : t;
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
          total = (isv ? 2u * (uint32_t)pages_in(first, BN) * 2u
                       : (uint32_t)(pages_in(first, KH) + pages_in(first + KH, KH)) * 4u) *
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
            if (!isv) {                             // 64 keys x 256 channels
              for (int bx = 0; bx < 4; ++bx)
                tma2_load_2d(smem_u32(dst + bx * (KH * 128)), own ? &tm_kr : &tm_kc, fb, part * 256 + bx * 64,
                             (int)row);
            } else {                                // 128 keys x 128 columns
              for (int bx = 0; bx < 2; ++bx)
                tma2_load_2d(smem_u32(dst + bx * (BN * 128)), own ? &tm_vr : &tm_vc, fb,
                             vh * DV + 128 * (int)rank + bx * 64, (int)row);
            }
          }
        } else {
          const int my_row = isv ? row_v : row_k;
          if (!isv) {
            const int pg = lane - 4 * (int)rank;    // lanes 4 rank .. 4 rank + 3 own the pages of this CTA's 64 keys
            if (pg >= 0 && pg < 4 && my_row >= 0)
              for (int bx = 0; bx < 4; ++bx)
                tma2_load_2d(smem_u32(dst + bx * (KH * 128) + pg * kPageSize * 128), &tm_kc, fb, part * 256 + bx * 64,
                             my_row);
          } else if (my_row >= 0) {
            for (int bx = 0; bx < 2; ++bx)
              tma2_load_2d(smem_u32(dst + bx * (BN * 128) + lane * kPageSize * 128), &tm_vc, fb,
                           vh * DV + 128 * (int)rank + bx * 64, my_row);
          }
        }
        __syncwarp();
        if (fix) {
          if (!__all_sync(kAll, mbar_wait(TAIL, tail_uses & 1, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          ++tail_uses;
          const int nz = BN - valid;
          for (int e = lane; e < 2 * nz * 8; e += 32) {
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
    // after a timeout too
    if (lane == 0 && leader) {
      int spare = 0;
      mbar_wait(Q_FULL, 0, &spare, kWaitNs);
      for (int jj = (j > NS ? j - NS : 0); jj < j; ++jj) mbar_wait(FULL(jj % NS), (jj / NS) & 1, &spare, kWaitNs);
    }
  } else if (warp == 5) {
    // ============================================================ MMA issuer (leader)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t ID_QK = idesc_bf16_f32(2 * BM, BN, 0, 0);
      constexpr uint32_t ID_PV = idesc_bf16_f32(2 * BM, DV, 0, 1);
      const uint32_t q_addr = smem_u32(sQ), ring_addr = smem_u32(ring);
      bool ok = mbar_wait(Q_FULL, 0, abort_flag, kWaitNs);
      tc_fence_after();
      int j = 0;
      for (int t = 0; t <= T && ok; ++t) {
        if (t < T) {
          const uint32_t sbuf = tmem + (uint32_t)((t & 1) * 128);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks, ++j) {
            const int slot = j % NS;
            if (!mbar_wait(FULL(slot), (j / NS) & 1, abort_flag, kWaitNs)) { ok = false; break; }
            tc_fence_after();
            const uint32_t kaddr = ring_addr + slot * SLOT;
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) {
              const uint64_t a = smem_desc(q_addr + (4 * ks + (kk >> 2)) * (BM * 128) + (kk & 3) * 32, 16, 1024, 2);
              const uint64_t bd = smem_desc(kaddr + (kk >> 2) * (KH * 128) + (kk & 3) * 32, 16, 1024, 2);
              mma_pair_ss(sbuf, a, bd, ID_QK, ks + kk > 0 ? 1u : 0u);
            }
            mma_commit_pair(EMPTY(slot));
          }
          if (!ok) break;
          mma_commit_pair(S_FULL(t & 1));
        }
        if (t >= 1) {
          const int u = t - 1, slot = j % NS;
          const uint32_t pbuf = tmem + (uint32_t)((u & 1) * 128), vaddr = ring_addr + slot * SLOT;
          if (!mbar_wait(FULL(slot), (j / NS) & 1, abort_flag, kWaitNs)) { ok = false; break; }
          tc_fence_after();
          for (int h = 0; h < 2 && ok; ++h) {
            if (!mbar_wait(P_FULL(u & 1, h), (u >> 1) & 1, abort_flag, kWaitNs)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int kq = 0; kq < BN / 32; ++kq) {
              const int kk = h * (BN / 32) + kq;
              const uint64_t bd = smem_desc(vaddr + kk * (16 * 128), BN * 128, 1024, 2);
              mma_pair_ts(tmem + 256, pbuf + kk * 8, bd, ID_PV, (u > 0 || kk > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          mma_commit_pair(EMPTY(slot));
          mma_commit_pair(O_DONE(u & 1));
          ++j;
        }
      }
      mma_commit_pair(FIN);
      int spare = 0;                                // (not abort_flag: this wait also follows a timeout)
      mbar_wait(FIN, 0, &spare, kWaitNs);
    }
  } else {
    // ============================================================ softmax and epilogue (own rows)
    const int r = tid;                              // row of the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t obuf = tmem + lane_base + 256;
    const float c2 = p.scale_log2;
    const int token = tok0 + r / G;                 // the row's place in its sequence
    const bool row_ok = r < p.rows_per_tile && token < n;
    const bool warp_live = __any_sync(kAll, row_ok);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < T; ++t) {
      if (!__all_sync(kAll, mbar_wait(S_FULL(t & 1), (t >> 1) & 1, abort_flag, kWaitNs))) { ok = false; break; }
      tc_fence_after();
      const uint32_t sbuf = tmem + lane_base + (uint32_t)((t & 1) * 128);
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
        const float m_new = fmaxf(m_ref, mx == -INFINITY ? -INFINITY : mx * c2);
        const bool first = m_ref == -INFINITY;
        const bool need = !first && m_new > m_ref + kRescaleThreshold;
        if (__any_sync(kAll, need)) {
          // O holds the tiles before this one once the last of their products is done
          const int u = t - 1;
          if (!__all_sync(kAll, mbar_wait(O_DONE(u & 1), (u >> 1) & 1, abort_flag, kWaitNs))) { ok = false; break; }
          tc_fence_after();
          const float alpha = need ? ex2(m_ref - m_new) : 1.f;
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            uint32_t rr[32];
            tmem_ld_x32(obuf + c, rr);
#pragma unroll
            for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st_x32(obuf + c, rr);
          }
          if (need) {
            l *= alpha;
            m_ref = m_new;
          }
        }
        if (first) m_ref = m_new;
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
          if (lane == 0) mbar_arrive_cluster(map_to_cta(P_FULL(t & 1, h), 0));
        }
        const float2 la = up2(fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3])));
        l += la.x + la.y;
      } else {
        // no row of this warp exists: whatever its lanes of P hold meets rows that are never read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(map_to_cta(P_FULL(t & 1, 0), 0));
          mbar_arrive_cluster(map_to_cta(P_FULL(t & 1, 1), 0));
        }
      }
    }
    const int u = T - 1;
    if (ok) ok = __all_sync(kAll, mbar_wait(O_DONE(u & 1), (u >> 1) & 1, abort_flag, kWaitNs));
    if (ok && warp_live) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      const int my_s = (Pt + token / BN) / p.chunk_tiles;     // the row's last split
      const bool split = my_s > 0, write = row_ok && s <= my_s;
      const int h = g * G + r % G;
      const int64_t at = split ? prompt_slot(o0 + token, h, s, p.Hq, p.splits) : (int64_t)(o0 + token) * p.Hq + h;
#pragma unroll 1
      for (int c = 0; c < DV; c += 32) {
        uint32_t rr[32];
        tmem_ld_x32(obuf + c, rr);
        if (!write) continue;
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(rr[e]) * inv;
        const int64_t to = at * D + vh * DV + c;
        if (!split && p.out_bf16) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + to);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>((split ? p.o_part : reinterpret_cast<float*>(p.out)) + to);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      if (write && split && vh == 0) p.ml_part[at] = make_float2(m_ref, l);
    }
  }

  // ---------------------------------------------------------------- teardown (pair)
  // The leader's last commit (FIN) reaches both CTAs after every earlier one:
  // once the peer has seen it, no arrive of the pair's products is under way
  // to its shared memory, and the cluster barrier keeps either CTA from
  // leaving before the other is done.
  if (T > 0 && warp == 5 && lane == 0 && rank != 0) {
    int spare = 0;
    mbar_wait(FIN, 0, &spare, kWaitNs);
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(p.status, TV_DEV_TIMEOUT);
  cluster_sync_relaxed();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

bool encode(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const PromptParams& p, int64_t units, cudaStream_t st) {
  CUtensorMap mq, mkc, mvc, mkr, mvr;
  const cuuint64_t row_bytes = (cuuint64_t)D * 2;
  {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.rows};
    cuuint64_t strides[2] = {row_bytes, row_bytes * p.Hq};
    cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(BM / p.G)};
    if (!encode(&mq, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const cuuint64_t strides[1] = {row_bytes};
  {
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)p.Hkv * p.rows};
    cuuint32_t kbox[2] = {64, KH}, vbox[2] = {64, BN};
    if (!encode(&mkr, p.k_rows, 2, dims, strides, kbox) || !encode(&mvr, p.v_rows, 2, dims, strides, vbox))
      return cudaErrorInvalidValue;
  }
  mkc = mkr;                                        // no prefix: never read
  mvc = mvr;
  if (p.max_prefix > 0) {
    cuuint64_t dims[2] = {(cuuint64_t)D, p.paged ? (cuuint64_t)p.num_pages * p.Hkv * kPageSize
                                                 : (cuuint64_t)p.B * p.Hkv * p.capacity};
    cuuint32_t kbox[2] = {64, (cuuint32_t)(p.paged ? kPageSize : KH)};
    cuuint32_t vbox[2] = {64, (cuuint32_t)(p.paged ? kPageSize : BN)};
    if (!encode(&mkc, p.k_cache, 2, dims, strides, kbox) || !encode(&mvc, p.v_cache, 2, dims, strides, vbox))
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
