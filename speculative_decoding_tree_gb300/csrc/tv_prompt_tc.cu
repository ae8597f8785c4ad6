// Causal prompt attention on tcgen05, bf16, head_dim 128: two query tiles a CTA.
//
// A unit is 2 x 128 query rows (token, group head) of one sequence and KV
// head; the two tiles share every K and V tile that comes in.  While the
// softmax of one tile works on its scores, the tensor cores multiply for the
// other: S_w(t) = Q_w K(t)^T into 128 columns of tensor memory, the softmax
// warps write the weights P_w(t) as bf16 over them, O_w += P_w(t) V(t).  The
// instructions are issued O_0(t), S_0(t + 1), O_1(t), S_1(t + 1), so each
// softmax has the time of two products of the other tile; one thread a row
// keeps the running maximum and sum, no exchange.  A weight is rounded to bf16
// (2^-8 of it at most) because the matrix unit multiplies equal types; the sum
// that divides keeps the fp32 weights.  A score buffer is refilled
// only after the weights in it were multiplied (instructions of one thread
// run in order), and the commit that hands S_w(t + 1) over covers O_w(t), so
// the row's accumulator stands still while its softmax may rescale it.
//
//   warps 0-3, 4-7  softmax and epilogue of tile 0 and 1
//   warp 8          TMA producer: Q, then K(0), V(0), K(1), V(1), ... in 32 KB
//                   slots (a paged cache in boxes of 16 rows)
//   warp 9          owns tensor memory; the warp runs the issue loop together and
//                   one lane's instructions are the products: operands then
//                   stay in uniform registers (a lane alone: 1.63 ms where this
//                   takes 1.27 for 16384 rows x 32 heads)
// Every wait is bounded (1 s); on a timeout the CTA raises TV_DEV_TIMEOUT and
// every role leaves its loop.
#include <cuda.h>

#include "tc_ptx.cuh"
#include "tv_f32x2.cuh"
#include "tv_prompt.cuh"
#include "tv_tensormap.cuh"

namespace tv {
namespace {

using namespace tc;

constexpr int D = 128;
constexpr int BM = 128;                         // rows of a query tile
constexpr int BN = kPromptTile;                 // keys of a tile
constexpr uint32_t BOX_BYTES = BN * 128;        // 128 rows x 64 bf16
constexpr uint32_t SLOT_BYTES = 2 * BOX_BYTES;
constexpr int NS = 5;                           // ring slots
constexpr uint32_t kHeader = 3 * 1024, kUnitOfs = 1024;
constexpr uint32_t Q_BYTES = 2 * BM * D * 2;
constexpr uint32_t SMEM = kHeader + Q_BYTES + NS * SLOT_BYTES;
static_assert(SMEM <= 232448, "shared memory over the 227 KB per-block limit");
constexpr int kThreads = 384;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescaleThreshold = 8.0f;       // rescale O when the maximum grows by more than 2^8

constexpr int B_FULL = 0, B_EMPTY = NS, B_Q = 2 * NS, B_S = B_Q + 1, B_P = B_S + 2, B_O = B_P + 4, B_TAIL = B_O + 2,
              B_FIN = B_TAIL + 1, NBARS = B_FIN + 1;

__global__ void __launch_bounds__(kThreads, 1)
prompt_tc_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                 const __grid_constant__ CUtensorMap tm_kr, const __grid_constant__ CUtensorMap tm_vr) {
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_raw + NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  PromptUnit& s_unit = *reinterpret_cast<PromptUnit*>(smem_raw + kUnitOfs);
  uint8_t* sQ = smem_raw + kHeader;
  uint8_t* ring = sQ + Q_BYTES;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto FULL = [&](int i) { return bar(B_FULL + i); };
  auto EMPTY = [&](int i) { return bar(B_EMPTY + i); };
  auto S_FULL = [&](int w) { return bar(B_S + w); };
  auto P_FULL = [&](int w, int h) { return bar(B_P + 2 * w + h); };   // key half h of tile w's weights
  auto O_DONE = [&](int w) { return bar(B_O + w); };
  const uint32_t Q_FULL = bar(B_Q), TAIL = bar(B_TAIL), FIN = bar(B_FIN);

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
    mbar_init(Q_FULL, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(S_FULL(w), 1);
      mbar_init(P_FULL(w, 0), 4);
      mbar_init(P_FULL(w, 1), 4);
      mbar_init(O_DONE(w), 1);
    }
    mbar_init(TAIL, 1);
    mbar_init(FIN, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (p.rows_per_tile < BM) {
    // pad rows of the query tiles (G does not divide 128) hold zeros; the Q loads never write them
    const int pad = BM - p.rows_per_tile;
    for (int e = tid; e < 4 * pad * 8; e += kThreads) {
      const int box = e / (pad * 8), r = p.rows_per_tile + (e / 8) % pad, c = e % 8;
      *reinterpret_cast<uint4*>(sQ + box * (BM * 128) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
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
  const int s = blockIdx.x % p.splits;
  const int rest = blockIdx.x / p.splits;
  const int g = rest % p.Hkv;
  if (warp == 0) find_unit(p, rest / p.Hkv, &s_unit);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the unit's rows and tiles (the same in every thread)
  const int b = s_unit.b, G = p.G, o0 = s_unit.o0, n = s_unit.n;
  const int64_t P = s_unit.P;
  const int tile_tokens = p.unit_tokens >> 1, tok0 = s_unit.i * p.unit_tokens;   // first token of the unit
  const int Pt = (int)((P + BN - 1) / BN);
  const int t_begin = s * p.chunk_tiles;
  int Tw[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int first = tok0 + w * tile_tokens;
    const int all = first < n ? Pt + (min(n, first + tile_tokens) - 1) / BN + 1 : 0;
    Tw[w] = max(0, min(all - t_begin, p.chunk_tiles));
  }
  const int T = max(Tw[0], Tw[1]);

  if (T == 0) {
    // nothing for this CTA
  } else if (warp == 8) {
    // ============================================================ producer
    if (lane == 0) {
      const uint32_t tile_bytes = (uint32_t)p.rows_per_tile * 128u * 2u;
      mbar_expect_tx(Q_FULL, tile_bytes * ((Tw[0] > 0) + (Tw[1] > 0)));
      for (int w = 0; w < 2; ++w)
        if (Tw[w] > 0)
          for (int kb = 0; kb < 2; ++kb)
            tma_load_3d(smem_u32(sQ + (2 * w + kb) * (BM * 128)), &tm_q, Q_FULL, kb * 64, g * G,
                        o0 + tok0 + w * tile_tokens);
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
    int pid_a = page_id(0), pid_b = page_id(1);
    int j = 0, tail_uses = 0;
    bool ok = true;
    for (int t = 0; t < T && ok; ++t) {
      const int tt = t_begin + t;
      const bool own = tt >= Pt;
      const int64_t first = own ? (int64_t)(tt - Pt) * BN : (int64_t)tt * BN;
      const int valid = (int)min((int64_t)BN, (own ? (int64_t)n : P) - first);   // keys of the tile that exist
      const int my_row = page_row(t, pid_a);
      pid_a = pid_b;
      pid_b = page_id(t + 2);
      for (int kind = 0; kind < 2 && ok; ++kind, ++j) {      // 0: K, 1: V
        const bool fix = kind == 1 && valid < BN;   // V rows past the end become zeros: their weights are
        const int slot = j % NS, use = j / NS;
        if (use > 0 && !__all_sync(kAll, mbar_wait(EMPTY(slot), (use - 1) & 1, abort_flag, kWaitNs))) {
          ok = false;
          break;
        }
        uint8_t* dst = ring + slot * SLOT_BYTES;
        const uint32_t fb = fix ? TAIL : FULL(slot);
        if (own || !p.paged) {
          if (lane == 0) {
            mbar_expect_tx(fb, SLOT_BYTES);
            const CUtensorMap* m = own ? (kind == 0 ? &tm_kr : &tm_vr) : (kind == 0 ? &tm_kc : &tm_vc);
            const int64_t row = own ? (int64_t)g * p.rows + o0 + first : ((int64_t)b * p.Hkv + g) * p.capacity + first;
            for (int bx = 0; bx < 2; ++bx) tma_load_2d(smem_u32(dst + bx * BOX_BYTES), m, fb, bx * 64, (int)row);
          }
        } else {
          const CUtensorMap* m = kind == 0 ? &tm_kc : &tm_vc;
          const int npages = __popc(__ballot_sync(kAll, my_row >= 0));
          if (lane == 0) mbar_expect_tx(fb, (uint32_t)npages * 2u * (kPageSize * 128u));
          __syncwarp();
          if (my_row >= 0)
            for (int bx = 0; bx < 2; ++bx)
              tma_load_2d(smem_u32(dst + bx * BOX_BYTES + lane * kPageSize * 128), m, fb, bx * 64, my_row);
        }
        __syncwarp();
        if (fix) {
          if (!__all_sync(kAll, mbar_wait_landed(TAIL, tail_uses & 1, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          ++tail_uses;
          const int nz = BN - valid;
          for (int e = lane; e < 2 * nz * 8; e += 32) {
            const int bx = e / (nz * 8), r = valid + (e / 8) % nz, q16 = e % 8;
            *reinterpret_cast<uint4*>(dst + bx * BOX_BYTES + r * 128 + q16 * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(FULL(slot));
        }
      }
    }
    // drain: every copy this warp started has landed before the CTA exits, after a timeout too
    if (lane == 0) {
      int spare = 0;
      mbar_wait(Q_FULL, 0, &spare, kWaitNs);
      for (int jj = (j > NS ? j - NS : 0); jj < j; ++jj) mbar_wait(FULL(jj % NS), (jj / NS) & 1, &spare, kWaitNs);
    }
  } else if (warp == 9) {
    // ============================================================ MMA issuer (the whole warp, one lane's instructions)
    constexpr uint32_t ID_QK = idesc_bf16_f32(BM, BN, 0, 0);
    constexpr uint32_t ID_PV = idesc_bf16_f32(BM, D, 0, 1);
    constexpr uint32_t HI = desc_hi(1024, 2);
    const uint32_t q_lo = desc_lo(smem_u32(sQ), 16), k_lo = desc_lo(smem_u32(ring), 16),
                   v_lo = desc_lo(smem_u32(ring), BOX_BYTES);
    const uint32_t tm = __shfl_sync(kAll, tmem, 0);
    const int n0 = __shfl_sync(kAll, Tw[0], 0), n1 = __shfl_sync(kAll, Tw[1], 0), nt = max(n0, n1);
    const bool one = elect_one();
    auto wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(kAll, mbar_wait(bar, parity, abort_flag, kWaitNs)) != 0;
    };
    auto qk = [&](int w, int slot) {
      const uint32_t a = q_lo + w * (2 * BM * 128 / 16), bd = k_lo + slot * (SLOT_BYTES / 16);
      const uint32_t to = tm + (uint32_t)(w * 128);
      if (one) {
        mma_ss_lo<false>(to, a, bd, HI, ID_QK);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk)
          mma_ss_lo<true>(to, a + (kk >> 2) * (BM * 128 / 16) + (kk & 3) * 2, bd + (kk >> 2) * (BOX_BYTES / 16) + (kk & 3) * 2,
                          HI, ID_QK);
        mma_commit(S_FULL(w));
      }
    };
    bool ok = wait(Q_FULL, 0) && wait(FULL(0), 0);
    tc_fence_after();
    if (ok) {
      if (n0 > 0) qk(0, 0);
      if (n1 > 0) qk(1, 0);
      if (one) mma_commit(EMPTY(0));
    }
    int vs = 1, vp = 0;                             // V(t)'s slot and phase; K(t + 1) follows it
    for (int t = 0; t < nt && ok; ++t) {
      int ks = vs + 1, kp = vp;
      if (ks == NS) {
        ks = 0;
        kp ^= 1;
      }
      ok = wait(FULL(vs), vp) && (t + 1 >= nt || wait(FULL(ks), kp));
      if (!ok) break;
      tc_fence_after();
      const uint32_t bd = v_lo + vs * (SLOT_BYTES / 16);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int nw = w == 0 ? n0 : n1;
        if (t < nw) {
          const uint32_t to = tm + 256 + (uint32_t)(w * D), pa = tm + (uint32_t)(w * 128);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && wait(P_FULL(w, h), t & 1);
            if (!ok) break;
            tc_fence_after();
            if (one) {
#pragma unroll
              for (int kq = 0; kq < BN / 32; ++kq) {
                const int kk = h * (BN / 32) + kq;
                if (kk == 0 && t == 0) mma_ts_lo<false>(to, pa, bd, HI, ID_PV);
                else mma_ts_lo<true>(to, pa + kk * 8, bd + kk * (16 * 128 / 16), HI, ID_PV);
              }
            }
          }
          if (!ok) break;
          if (one && t == nw - 1) mma_commit(O_DONE(w));
        }
        if (one && w == 1) mma_commit(EMPTY(vs));
        if (t + 1 < nw) qk(w, ks);
      }
      if (!ok) break;
      if (one && t + 1 < nt) mma_commit(EMPTY(ks));
      vs = ks + 1;
      vp = kp;
      if (vs == NS) {
        vs = 0;
        vp ^= 1;
      }
    }
    // every product issued has finished before tensor memory is freed
    if (one) mma_commit(FIN);
    int spare = 0;                                  // (not abort_flag: this wait also follows a timeout)
    mbar_wait(FIN, 0, &spare, kWaitNs);
    __syncwarp();
  } else if (warp < 8) {
    // ============================================================ softmax and epilogue
    const int w = warp >> 2;
    const int myT = Tw[w];
    const int r = (warp & 3) * 32 + lane;           // row of the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sbuf = tmem + lane_base + (uint32_t)(w * 128);
    const uint32_t obuf = tmem + lane_base + 256 + (uint32_t)(w * D);
    const float c2 = p.scale_log2;
    const int token = tok0 + w * tile_tokens + r / G;   // the row's place in its sequence
    const bool row_ok = r < p.rows_per_tile && token < n;
    const bool warp_live = __any_sync(kAll, row_ok);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < myT; ++t) {
      if (!__all_sync(kAll, mbar_wait(S_FULL(w), t & 1, abort_flag, kWaitNs))) { ok = false; break; }
      tc_fence_after();
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
          const float alpha = need ? ex2(m_ref - m_new) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t rr[16];
            tmem_ld_x16(obuf + c, rr);
#pragma unroll
            for (int e = 0; e < 16; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st_x16(obuf + c, rr);
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
          if (lane == 0) mbar_arrive(P_FULL(w, h));
        }
        const float2 la = up2(fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3])));
        l += la.x + la.y;
      } else {
        // no row of this warp exists: whatever its lanes of P hold meets rows that are never read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(P_FULL(w, 0));
          mbar_arrive(P_FULL(w, 1));
        }
      }
    }
    if (ok && myT > 0) ok = __all_sync(kAll, mbar_wait(O_DONE(w), 0, abort_flag, kWaitNs));
    if (ok && myT > 0) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      // Rows go out through the query tile's shared memory, which no product reads any more: a thread stages its row
      // 16 bytes at a time (piece c at c ^ (row & 7)), then 16 lanes store a row of 256 bytes together.  (Each thread
      // storing its own row took 3 us of a CTA.)
      uint8_t* stage = sQ + w * 2 * (BM * 128) + (warp & 3) * (32 * 256);
      const int my_s = (Pt + token / BN) / p.chunk_tiles;     // the row's last split
      const bool wide = !p.out_bf16 || my_s > 0;    // fp32: partials, or the output's type
      const int64_t slot = my_s > 0 ? prompt_slot(o0 + token, g * G + r % G, s, p.Hq, p.splits)
                                    : (int64_t)(o0 + token) * p.Hq + g * G + r % G;
      const bool write = row_ok && s <= my_s;
      // (bf16 rows and fp32 ones may meet in a warp: both forms run where both occur)
      const unsigned any_wide = __ballot_sync(kAll, write && wide), any_slim = __ballot_sync(kAll, write && !wide);
      auto flush = [&](unsigned rows, char* base, int64_t row_bytes, int col_bytes) {
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int rr = 2 * i + (lane >> 4), c = lane & 15;
          const int64_t at = __shfl_sync(kAll, slot, rr);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 256 + ((c ^ (rr & 7)) << 4));
          if (rows >> rr & 1u) *reinterpret_cast<uint4*>(base + at * row_bytes + col_bytes + c * 16) = v;
        }
        __syncwarp();
      };
      if (any_slim) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t rr[32];
          tmem_ld_x32(obuf + c, rr);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 v;
            uint32_t* vw = &v.x;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              vw[q] = pack_bf16(__uint_as_float(rr[8 * e + 2 * q]) * inv, __uint_as_float(rr[8 * e + 2 * q + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + lane * 256 + (((c / 8 + e) ^ (lane & 7)) << 4)) = v;
          }
        }
        flush(any_slim, reinterpret_cast<char*>(p.out), D * 2, 0);
      }
      if (any_wide) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {            // 64 columns at a time
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t rr[32];
            tmem_ld_x32(obuf + hf * 64 + c, rr);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = make_float4(__uint_as_float(rr[4 * e]) * inv, __uint_as_float(rr[4 * e + 1]) * inv,
                                           __uint_as_float(rr[4 * e + 2]) * inv, __uint_as_float(rr[4 * e + 3]) * inv);
              *reinterpret_cast<float4*>(stage + lane * 256 + (((c / 4 + e) ^ (lane & 7)) << 4)) = v;
            }
          }
          const unsigned parts = __ballot_sync(kAll, write && my_s > 0);
          if (parts) flush(parts, reinterpret_cast<char*>(p.o_part), D * 4, hf * 256);
          if (any_wide & ~parts) flush(any_wide & ~parts, reinterpret_cast<char*>(p.out), D * 4, hf * 256);
        }
      }
      if (write && my_s > 0) p.ml_part[slot] = make_float2(m_ref, l);
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(p.status, TV_DEV_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool prompt_tc_supported(const tv_desc* d, int64_t rows) {
  const int64_t most = ((int64_t)1 << 31) - 1 - BN;  // TMA row coordinates are 32 bits
  const int G = d->num_q_heads / d->num_kv_heads;
  int64_t cache = d->page_size ? d->num_pages * d->num_kv_heads * kPageSize
                               : (int64_t)d->batch * d->num_kv_heads * d->capacity;
  if (d->max_prefix == 0) cache = 0;
  return d->dtype == TV_BF16 && G <= BM && cache <= most && rows * d->num_kv_heads <= most;
}

cudaError_t launch_prompt_tc(const PromptParams& p, int64_t units, cudaStream_t st) {
  CUtensorMap mq, mkc, mvc, mkr, mvr;
  const cuuint64_t row_bytes = (cuuint64_t)D * 2;
  {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.rows};
    cuuint64_t strides[2] = {row_bytes, row_bytes * p.Hq};
    cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(BM / p.G)};
    if (!encode_rows(&mq, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)p.Hkv * p.rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {64, BN};
    if (!encode_rows(&mkr, p.k_rows, 2, dims, strides, box) || !encode_rows(&mvr, p.v_rows, 2, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  mkc = mkr;                                        // no prefix: never read
  mvc = mvr;
  if (p.max_prefix > 0) {
    const cuuint64_t rows = p.paged ? (cuuint64_t)p.num_pages * p.Hkv * kPageSize
                                    : (cuuint64_t)p.B * p.Hkv * p.capacity;
    cuuint64_t dims[2] = {(cuuint64_t)D, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {64, (cuuint32_t)(p.paged ? kPageSize : BN)};
    if (!encode_rows(&mkc, p.k_cache, 2, dims, strides, box) || !encode_rows(&mvc, p.v_cache, 2, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  const cudaError_t e = ensure_max_dynamic_smem<prompt_tc_kernel>((int)SMEM);
  if (e != cudaSuccess) return e;
  return launch_dep(prompt_tc_kernel, dim3((unsigned)(units * p.Hkv * p.splits)), dim3(kThreads), SMEM, st, p, mq, mkc,
                    mvc, mkr, mvr);
}

}  // namespace tv
