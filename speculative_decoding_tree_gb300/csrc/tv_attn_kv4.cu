// tcgen05 split-KV tree-verify attention over a 4-bit cache (tree_kv4.h):
// bf16 queries and tree K/V, fp32 accumulation and softmax, head_dim 128, 256
// or 512.
//
// The method is flash-decode with a tree mask: a unit of work (sequence, KV
// head, tile of up to 64 query rows, chunk of keys) leaves a normalised
// partial output with its reference exponent m and its sum l, and the
// log-sum-exp merge joins the chunks.
//
// Both products are taken transposed, so that the cache's values are the A
// operand and go from registers into tensor memory, never through shared
// memory, and so that a few query rows cost a few columns instead of a
// 128-row tile:
//   S^T [128 keys x 64 rows]     = K  [keys x d]        Q^T   (A: tensor memory, B: Q in shared memory)
//   O^T [128 channels x 64 rows] += V^T [channels x keys] P^T  (A: tensor memory, B: P in shared memory)
// A lane of an A operand is a key of K and a channel of V: the cache's K
// blocks hold a key's 32 channels in 16 bytes, its V blocks a channel's 16
// keys in 8, so a thread expands whole words into consecutive columns.
//
// Expansion.  A word's value pair (bits 4 j and 16 + 4 j) is masked into two
// bf16 numbers 128 + u; K's is then one fused multiply-add,
// (128 + u) s - 136 s = (u - 8) s, exact because s has 4 significant bits; V's
// is u - 8, exact, and the position's V scale multiplies the softmax weight
// before it is rounded to bf16.
//
// Softmax.  A thread owns one key and up to 32 rows.  The exponent reference
// of a row need not be its maximum: any reference within 2^60 of it gives the
// same weights, since bf16 weights and fp32 sums keep their relative precision
// there.  So the first key's score serves, and only a score above the
// reference by more than 60 (log2) takes the true column maximum and rescales
// O.  Tiles whose mask hides keys from some rows start from the true maximum.
//
// Warps: 0 bulk loads, 1 MMA issue, 2 the list of units, 4-11 expansion (two
// groups of 128 lanes), 12-19 softmax and epilogue (two groups, each half of
// the rows).  The grid is persistent: CTA c takes units c, c + grid, ..., and
// loads and expands the next unit's keys while it finishes the last one.
//
// Every mbarrier wait is bounded (1 s); on a timeout the CTA raises
// TV_DEV_TIMEOUT, waits for its own copies and MMAs, frees tensor memory and
// returns.
#include <cuda.h>

#include <mutex>

#include "tc_ptx.cuh"
#include "tv_kv4.cuh"

namespace tv {
namespace {

using namespace tc;

constexpr int BK = 128;                          // keys per tile
constexpr int BN = 64;                           // query rows per tile
constexpr int kBlocks = BK / kPageSize;          // cache blocks per tile
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kHeadroom = 60.0f;               // log2: a weight above 2^60 moves the reference
constexpr int kExpandWarps = 8, kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (4 + kExpandWarps + kSoftmaxWarps);
constexpr int kUnits = 4;                        // units listed ahead
constexpr int kConsumers = 2 + kExpandWarps + kSoftmaxWarps;
constexpr uint32_t kHeader = 4096;
constexpr uint32_t P_BYTES = BK * 128;           // 128 keys x 64 bf16

template <int D>
struct Cfg {
  static constexpr int CPT = D / 128;                       // 128-channel chunks of a tile
  static constexpr int KB = kv4::k_block_bytes(D), VB = kv4::v_block_bytes(D);
  static constexpr int NK = D == 128 ? 8 : (D == 256 ? 3 : 2);
  static constexpr int NV = D == 128 ? 8 : (D == 256 ? 3 : 1);
  static constexpr int NQ = D == 512 ? 1 : 2;               // query tiles in shared memory
  static constexpr int NO = D == 128 ? 2 : 1;               // output accumulators
  static constexpr int NA = D == 512 ? 2 : 4;               // A operands in tensor memory (64 columns)
  static constexpr uint32_t Q_BYTES = BN * D * 2;
  static constexpr uint32_t K_SLOT = kBlocks * KB, V_SLOT = kBlocks * VB;
  static constexpr uint32_t SMEM = kHeader + NQ * Q_BYTES + 2 * P_BYTES + NK * K_SLOT + NV * V_SLOT;
  // tensor memory columns: outputs, two score tiles, A operands
  static constexpr uint32_t T_S = NO * CPT * BN, T_A = T_S + 2 * BN;
  static constexpr int NBARS = 2 * (NK + NV + NA + NQ + kUnits) + 8 + NO + 1;
  static_assert(T_A + NA * 64 <= 512, "tensor memory");
  static_assert(SMEM <= 232448, "shared memory over the 227 KB per-block limit");
  static_assert(NBARS * 8 <= 512, "barriers overflow their area");
};

struct Unit {
  int64_t P, k_begin, s0, w0;
  int b, g, rt, s, o0, n, nch;
  int T;                                         // tiles (the tree's included); < 0: no more units
  int npt, tail;                                 // prefix tiles; keys of the last one
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// pair j of a word as two bf16 numbers 128 + u
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int j) { return ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u; }

constexpr uint32_t kMinus136 = 0xC308C308u, kOne = 0x3F803F80u, kZero = 0x80008000u;   // bf16 pairs (kZero: -0)

__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n"
      :
      : "r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld_x8(uint32_t a, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n"
      "tcgen05.wait::st.sync.aligned;\n" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[8]) { tmem_ld_x8(a, r); }
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[16]) { tmem_ld_x16(a, r); }
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[32]) { tmem_ld_x32(a, r); }
__device__ __forceinline__ void st_cols(uint32_t a, const uint32_t (&r)[8]) { tmem_st_x8(a, r); }
__device__ __forceinline__ void st_cols(uint32_t a, const uint32_t (&r)[16]) { tmem_st_x16(a, r); }
__device__ __forceinline__ void st_cols(uint32_t a, const uint32_t (&r)[32]) { tmem_st_x32(a, r); }

// barrier `id` of one softmax group (128 threads), and the OR of a predicate over it
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_or(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "bar.red.or.pred q, %2, 128, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

struct MaxOp { static __device__ __forceinline__ float f(float a, float b) { return fmaxf(a, b); } };
struct SumOp { static __device__ __forceinline__ float f(float a, float b) { return a + b; } };

// Reduces HC values per lane over the warp: lane L returns column L & (HC - 1).
template <typename Op, int HC>
__device__ __forceinline__ float reduce_columns(float (&v)[HC]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = HC / 2; n >= 1; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = Op::f(keep, __shfl_xor_sync(0xffffffffu, send, n));
    }
  }
#pragma unroll
  for (int off = HC; off < 32; off <<= 1) v[0] = Op::f(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
  return v[0];
}

// shared memory: barriers (0..511), then these
struct Shared {
  uint32_t tmem;
  int abort_flag;
  Unit units[kUnits];
  alignas(16) float nm[2][32];                   // -reference of each row (-inf: not a row)
  uint32_t none[2];                              // rows without a reference yet
  float red[2][4][32];                           // per-warp column results
  float inv[2][32];
  uint64_t anc[2][32];
  int dep[2][32];
};
static_assert(512 + sizeof(Shared) <= kHeader, "header");

template <int D>
struct Bars {
  using C = Cfg<D>;
  uint32_t base;
  __device__ __forceinline__ uint32_t at(int i) const { return base + 8u * (uint32_t)i; }
  __device__ __forceinline__ uint32_t k_full(int i) const { return at(i); }
  __device__ __forceinline__ uint32_t k_empty(int i) const { return at(C::NK + i); }
  __device__ __forceinline__ uint32_t v_full(int i) const { return at(2 * C::NK + i); }
  __device__ __forceinline__ uint32_t v_empty(int i) const { return at(2 * C::NK + C::NV + i); }
  static constexpr int a0 = 2 * (C::NK + C::NV);
  __device__ __forceinline__ uint32_t a_full(int i) const { return at(a0 + i); }
  __device__ __forceinline__ uint32_t a_empty(int i) const { return at(a0 + C::NA + i); }
  static constexpr int q0 = a0 + 2 * C::NA;
  __device__ __forceinline__ uint32_t q_full(int i) const { return at(q0 + i); }
  __device__ __forceinline__ uint32_t q_empty(int i) const { return at(q0 + C::NQ + i); }
  static constexpr int u0 = q0 + 2 * C::NQ;
  __device__ __forceinline__ uint32_t u_full(int i) const { return at(u0 + i); }
  __device__ __forceinline__ uint32_t u_empty(int i) const { return at(u0 + kUnits + i); }
  static constexpr int s0 = u0 + 2 * kUnits;
  __device__ __forceinline__ uint32_t s_full(int i) const { return at(s0 + i); }
  __device__ __forceinline__ uint32_t s_empty(int i) const { return at(s0 + 2 + i); }
  __device__ __forceinline__ uint32_t p_full(int i) const { return at(s0 + 4 + i); }
  __device__ __forceinline__ uint32_t pv_done(int i) const { return at(s0 + 6 + i); }
  static constexpr int o0 = s0 + 8;
  __device__ __forceinline__ uint32_t o_empty(int i) const { return at(o0 + i); }
  __device__ __forceinline__ uint32_t fin() const { return at(o0 + C::NO); }
};

template <int D, bool WIN>
struct Softmax {
  using C = Cfg<D>;
  const AttnParams& p;
  const Bars<D>& bars;
  Shared& sh;
  uint8_t* sP;
  const uint8_t* sV;
  uint32_t tmem;
  int tiles = 0, vuse = 0, unit = 0;             // running counts over the units

  // One unit: HC rows per group, one key per thread.  Returns false (on every
  // thread of the group) when a wait gave up.
  template <int HC>
  __device__ bool run(const Unit& u) {
    constexpr unsigned kAll = 0xffffffffu;
    volatile int* abort_flag = &sh.abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp = (warp - 4 - kExpandWarps) >> 2, key = (warp & 3) * 32 + lane;
    const int bar_id = 1 + grp, c0 = grp * HC, m0 = u.rt * p.rows_per_tile;
    const int live = min(p.rows_per_tile, u.n * p.G - m0);          // rows of the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c2 = p.scale_log2;
    const int64_t first_pos = WIN ? u.P - p.window + 1 : 0;
    const bool has_tree = u.T > u.npt;
    float* nm = sh.nm[grp];
    if (has_tree || WIN) {
      if (key < HC) {
        const int m = m0 + c0 + key;
        const bool ok = c0 + key < live;
        sh.anc[grp][key] = ok ? p.anc[u.o0 + m / p.G] : 0ull;
        if (WIN) sh.dep[grp][key] = ok ? p.depth[u.o0 + m / p.G] : 0;
      }
    }
    int key_dep = 0;
    if (WIN && has_tree && key < u.n) key_dep = p.depth[u.o0 + key];
    if (key < HC) nm[key] = c0 + key < live ? 0.f : -INFINITY;
    if (key == 0) {
      const int mine = max(0, min(HC, live - c0));
      sh.none[grp] = mine == 32 ? 0xffffffffu : (1u << mine) - 1u;
    }
    group_sync(bar_id);
    float l[HC];
#pragma unroll
    for (int j = 0; j < HC; ++j) l[j] = 0.f;
    const uint32_t obase = tmem + lane_base + (uint32_t)((unit % C::NO) * C::CPT * BN + c0);

    for (int t = 0; t < u.T; ++t) {
      const int x = tiles + t, buf = x & 1;
      const bool tree = t == u.npt;
      bool ok = __all_sync(kAll, mbar_wait(bars.s_full(buf), (x >> 1) & 1, abort_flag, kWaitNs));
      // this tile's V scale of the thread's key
      float sv = 1.f;
      if (!tree) {
        const int vs = (vuse + t) % C::NV;
        ok = __all_sync(kAll, ok && mbar_wait(bars.v_full(vs), ((vuse + t) / C::NV) & 1, abort_flag, kWaitNs)) && ok;
        const uint8_t* blk = sV + vs * C::V_SLOT + (key >> 4) * C::VB;
        sv = kv4::scale_of(blk[kv4::v_scale(D, key & 15)]);
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.v_empty(vs));
      }
      // the P buffer is free when the product two tiles back is done
      if (x >= 2) ok = __all_sync(kAll, ok && mbar_wait(bars.pv_done(buf), ((x - 2) >> 1) & 1, abort_flag, kWaitNs)) && ok;
      tc_fence_after();
      float s[HC];
      {
        uint32_t r[HC];
        ld_cols(tmem + lane_base + C::T_S + (uint32_t)(buf * BN + c0), r);
#pragma unroll
        for (int j = 0; j < HC; ++j) s[j] = __uint_as_float(r[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.s_empty(buf));

      // what the thread's key shows to the rows
      bool by_row = tree;
      if (!tree) {
        const bool in = t < u.npt - 1 || key < u.tail;
        int64_t pos = 0;
        if (WIN) {
          const int64_t v = u.k_begin + (int64_t)t * BK;
          const int64_t p0 = v < u.s0 ? v : v - u.s0 + u.w0;
          by_row = p0 < u.P + kMaxNodes - p.window;
          pos = p0 + key;
        }
        if (by_row) {
#pragma unroll
          for (int j = 0; j < HC; ++j)
            if (!in || !(pos < p.sinks || pos >= first_pos + sh.dep[grp][j])) s[j] = -INFINITY;
        } else if (!in) {
#pragma unroll
          for (int j = 0; j < HC; ++j) s[j] = -INFINITY;
        }
      } else {
#pragma unroll
        for (int j = 0; j < HC; ++j) {
          bool vis = key < kMaxNodes && ((sh.anc[grp][j] >> (key & 63)) & 1ull);
          if (WIN) vis = vis && (u.P + key_dep < p.sinks || sh.dep[grp][j] - (int64_t)key_dep < p.window);
          if (!vis) s[j] = -INFINITY;
        }
      }

      if (t == 0 && !by_row) {
        // every row sees key 0: its scores are the references
        if (key == 0) {
#pragma unroll
          for (int j = 0; j < HC; ++j)
            if (c0 + j < live) nm[j] = -s[j] * c2;
          sh.none[grp] = 0;
        }
        group_sync(bar_id);
      }
      float xm = -INFINITY;
#pragma unroll
      for (int j4 = 0; j4 < HC / 4; ++j4) {
        const float4 n4 = reinterpret_cast<const float4*>(nm)[j4];
        s[4 * j4] = fmaf(s[4 * j4], c2, n4.x);
        s[4 * j4 + 1] = fmaf(s[4 * j4 + 1], c2, n4.y);
        s[4 * j4 + 2] = fmaf(s[4 * j4 + 2], c2, n4.z);
        s[4 * j4 + 3] = fmaf(s[4 * j4 + 3], c2, n4.w);
        xm = fmaxf(fmaxf(fmaxf(xm, s[4 * j4]), fmaxf(s[4 * j4 + 1], s[4 * j4 + 2])), s[4 * j4 + 3]);
      }
      if (group_or(bar_id, !ok || xm > kHeadroom || sh.none[grp] != 0)) {
        // a wait gave up, a score is far above its reference, or a row has none yet
        bool good = ok;
        if (t > 0) good = __all_sync(kAll, good && mbar_wait(bars.pv_done((x - 1) & 1), ((x - 1) >> 1) & 1, abort_flag, kWaitNs));
        tc_fence_after();
        float v[HC];
#pragma unroll
        for (int j = 0; j < HC; ++j) v[j] = s[j];
        const float top = reduce_columns<MaxOp>(v);
        if (lane < HC) sh.red[grp][warp & 3][lane] = top;
        if (group_or(bar_id, !good)) return false;
        // column maxima relative to the present reference; a row moves when
        // it has no reference or its scores are above it
        const uint32_t none = sh.none[grp];
        float d = 0.f;                                             // how far row `lane` moves
        if (lane < HC && c0 + lane < live) {
          const float mx = fmaxf(fmaxf(sh.red[grp][0][lane], sh.red[grp][1][lane]),
                                 fmaxf(sh.red[grp][2][lane], sh.red[grp][3][lane]));
          if (mx != -INFINITY && (((none >> lane) & 1u) || mx > 0.f)) d = mx;
          // a row without a reference has neither weights nor a sum yet
          if (mx != -INFINITY && ((none >> lane) & 1u)) d = mx;
        }
        const uint32_t seen = __ballot_sync(kAll, lane < HC && d != 0.f);
        const float alpha_own = ((none >> lane) & 1u) ? 1.f : ex2(-d);
        float al[HC];
#pragma unroll
        for (int j = 0; j < HC; ++j) {
          const float dj = __shfl_sync(kAll, d, j);
          al[j] = __shfl_sync(kAll, alpha_own, j);
          s[j] -= dj;
          l[j] *= al[j];
        }
        if (t > 0 && seen) {
#pragma unroll 1
          for (int c = 0; c < C::CPT; ++c) {
            uint32_t r[HC];
            ld_cols(obase + c * BN, r);
#pragma unroll
            for (int j = 0; j < HC; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * al[j]);
            st_cols(obase + c * BN, r);
          }
          tc_fence_before();
        }
        const bool found = lane < HC && c0 + lane < live &&
                           fmaxf(fmaxf(sh.red[grp][0][lane & (HC - 1)], sh.red[grp][1][lane & (HC - 1)]),
                                 fmaxf(sh.red[grp][2][lane & (HC - 1)], sh.red[grp][3][lane & (HC - 1)])) != -INFINITY;
        const uint32_t have = __ballot_sync(kAll, found);
        group_sync(bar_id);                                        // every warp has read nm, none and red
        if ((warp & 3) == 0) {
          if (lane < HC) nm[lane] -= d;
          if (lane == 0) sh.none[grp] = none & ~have;
        }
        group_sync(bar_id);
      }
      // weights, sums, and the V-scaled weights as bf16 into the P tile:
      // key row of 128 bytes, 16-byte chunk c at c ^ (key & 7)
      uint8_t* prow = sP + buf * P_BYTES + key * 128;
#pragma unroll
      for (int j8 = 0; j8 < HC / 8; ++j8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = ex2(s[8 * j8 + 2 * e]), p1 = ex2(s[8 * j8 + 2 * e + 1]);
          l[8 * j8 + 2 * e] += p0;
          l[8 * j8 + 2 * e + 1] += p1;
          w[e] = pack_bf16(p0 * sv, p1 * sv);
        }
        *reinterpret_cast<uint4*>(prow + (((c0 / 8 + j8) ^ (key & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.p_full(buf));
    }

    // epilogue: the sums over the keys, then the rows of O / l
    const int x = tiles + u.T - 1;
    const bool ok = __all_sync(kAll, mbar_wait(bars.pv_done(x & 1), (x >> 1) & 1, abort_flag, kWaitNs));
    tc_fence_after();
    const float sum = reduce_columns<SumOp>(l);
    if (lane < HC) sh.red[grp][warp & 3][lane] = sum;
    if (group_or(bar_id, !ok)) return false;
    const bool direct = p.out != nullptr && u.nch == 1;
    const int64_t slot0 = partial_slot(u.s, u.b, u.g, u.rt, c0, p.Hkv, p.row_tiles, p.tile_stride, p.splits);
    if (key < HC) {
      const float L = (sh.red[grp][0][key] + sh.red[grp][1][key]) + (sh.red[grp][2][key] + sh.red[grp][3][key]);
      sh.inv[grp][key] = L > 0.f ? 1.f / L : 0.f;
      if (!direct && c0 + key < live)
        p.ml_part[slot0 + (int64_t)key * p.splits] =
            make_float2(((sh.none[grp] >> key) & 1u) ? -INFINITY : -nm[key], L);
    }
    group_sync(bar_id);
    const int rows = min(HC, live - c0);
#pragma unroll 1
    for (int c = 0; c < C::CPT; ++c) {
      uint32_t r[HC];
      ld_cols(obase + c * BN, r);
      const int ch = c * 128 + key;                                // TMEM lane = channel of the chunk
      if (direct) {
#pragma unroll
        for (int j = 0; j < HC; ++j) {
          if (j >= rows) break;
          const int m = m0 + c0 + j;
          const int64_t e = ((int64_t)(u.o0 + m / p.G) * p.Hq + u.g * p.G + m % p.G) * D + ch;
          const float v = __uint_as_float(r[j]) * sh.inv[grp][j];
          if (p.out_bf16)
            reinterpret_cast<__nv_bfloat16*>(p.out)[e] = __float2bfloat16_rn(v);
          else
            reinterpret_cast<float*>(p.out)[e] = v;
        }
      } else {
        float* dst = p.o_part + slot0 * D + ch;
#pragma unroll
        for (int j = 0; j < HC; ++j) {
          if (j >= rows) break;
          dst[(int64_t)j * p.splits * D] = __uint_as_float(r[j]) * sh.inv[grp][j];
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.o_empty(unit % C::NO));
    group_sync(bar_id);                                            // inv, nm and red are free
    tiles += u.T;
    vuse += u.npt;
    ++unit;
    return true;
  }
};

template <int D, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
tv_attn_kv4_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap tm_q) {
  using C = Cfg<D>;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw + 512);
  uint8_t* sQ = smem_raw + kHeader;
  uint8_t* sP = sQ + C::NQ * C::Q_BYTES;
  uint8_t* sK = sP + 2 * P_BYTES;
  uint8_t* sV = sK + C::NK * C::K_SLOT;
  Bars<D> bars{smem_u32(smem_raw)};
  volatile int* abort_flag = &sh.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // the swizzled tiles need the dynamic shared window to start 1 KB aligned
  if (smem_u32(smem_raw) & 1023u) {
    dep_wait();
    if (tid == 0) set_status(p.status, TV_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(bars.k_full(i), 1);
      mbar_init(bars.k_empty(i), C::CPT * 4);                // four expansion warps a chunk
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(bars.v_full(i), 1);
      mbar_init(bars.v_empty(i), C::CPT * 4 + kSoftmaxWarps);
    }
    for (int i = 0; i < C::NA; ++i) {
      mbar_init(bars.a_full(i), 4);
      mbar_init(bars.a_empty(i), 1);
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(bars.q_full(i), 1);
      mbar_init(bars.q_empty(i), 1);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(bars.u_full(i), 1);
      mbar_init(bars.u_empty(i), kConsumers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.s_full(i), 1);
      mbar_init(bars.s_empty(i), kSoftmaxWarps);
      mbar_init(bars.p_full(i), kSoftmaxWarps);
      mbar_init(bars.pv_done(i), 1);
    }
    for (int i = 0; i < C::NO; ++i) mbar_init(bars.o_empty(i), kSoftmaxWarps);
    mbar_init(bars.fin(), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (p.rows_per_tile < BN) {
    // pad rows of the query tiles (G does not divide 64) hold zeros
    const int pad = BN - p.rows_per_tile;
    for (int e = tid; e < C::NQ * (D / 64) * pad * 8; e += kThreads) {
      const int kb = e / (pad * 8), r = p.rows_per_tile + (e / 8) % pad, c = e % 8;
      *reinterpret_cast<uint4*>(sQ + kb * (BN * 128) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  if (tid == 0) tma_prefetch_desc(&tm_q);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  dep_wait();
  dep_launch();

  // the next unit of this role (false: a wait gave up); the slot is released
  // once its fields are in registers
  int nu = 0;
  auto next_unit = [&](Unit& u) -> bool {
    const int i = nu % kUnits;
    if (!__all_sync(kAll, mbar_wait(bars.u_full(i), (nu / kUnits) & 1, abort_flag, kWaitNs))) return false;
    u = sh.units[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.u_empty(i));
    ++nu;
    return true;
  };

  if (warp == 2) {
    // ============================================================ units
    // Sequence b has KV heads x row tiles x chunks units (none when its rows
    // are invalid), numbered on from sequence b - 1's; 32 sequences at a time.
    int64_t base = 0, want = blockIdx.x;
    int w = 0;
    bool ok = true;
    auto put = [&](const Unit& u) {
      const int i = w % kUnits;
      if (w >= kUnits) ok = __all_sync(kAll, mbar_wait(bars.u_empty(i), (w / kUnits - 1) & 1, abort_flag, kWaitNs));
      if (!ok) return;
      if (lane == 0) {
        sh.units[i] = u;
        mbar_arrive(bars.u_full(i));
      }
      __syncwarp();
      ++w;
    };
    for (int b0 = 0; b0 < p.B && ok; b0 += 32) {
      const int b = b0 + lane;
      int o0 = 0, n = 0, nch = 0, rts = 0;
      int64_t P = 0, cnt = 0;
      KeyMap km{0, 0, 0};
      if (b < p.B) {
        const int64_t Praw = p.prefix_len[b];
        int32_t* st = blockIdx.x == 0 ? p.status : nullptr;
        if (seq_rows(p.node_offsets, b, p.R, p.max_nodes, st, &o0, &n)) {
          P = clamp_prefix(Praw, p.max_prefix, p.capacity);
          if (P != Praw) set_status(st, TV_DEV_BAD_PREFIX);
          km = key_map(P, WIN ? p.window : 0, p.sinks, p.map_tile);
          nch = num_chunks(km.len, p.chunk, p.tree_tile);
          rts = (n * p.G + p.rows_per_tile - 1) / p.rows_per_tile;
          cnt = (int64_t)p.Hkv * rts * nch;
        }
      }
      int64_t incl = cnt;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(kAll, incl, off);
        if (lane >= off) incl += o;
      }
      const int64_t total = __shfl_sync(kAll, incl, 31);
      while (ok && want < base + total) {
        const int src = __ffs(__ballot_sync(kAll, want < base + incl)) - 1;
        const int64_t before = __shfl_sync(kAll, incl - cnt, src);
        Unit u;
        u.b = b0 + src;
        u.o0 = __shfl_sync(kAll, o0, src);
        u.n = __shfl_sync(kAll, n, src);
        u.nch = __shfl_sync(kAll, nch, src);
        u.P = __shfl_sync(kAll, P, src);
        u.s0 = __shfl_sync(kAll, km.s0, src);
        u.w0 = __shfl_sync(kAll, km.w0, src);
        const int64_t len = __shfl_sync(kAll, km.len, src);
        const int rt_n = __shfl_sync(kAll, rts, src);
        const int64_t k = want - base - before;
        u.s = (int)(k % u.nch);
        u.rt = (int)(k / u.nch % rt_n);
        u.g = (int)(k / u.nch / rt_n);
        u.k_begin = (int64_t)u.s * p.chunk;
        const int64_t k_end = min(len, u.k_begin + p.chunk);
        u.npt = (int)((k_end - u.k_begin + BK - 1) / BK);
        if (u.npt < 0) u.npt = 0;
        u.tail = u.npt > 0 ? (int)(k_end - u.k_begin - (int64_t)(u.npt - 1) * BK) : BK;
        u.T = u.npt + (u.s == u.nch - 1 ? 1 : 0);
        put(u);
        want += gridDim.x;
      }
      base += total;
    }
    Unit end;
    end.T = -1;
    if (ok) put(end);
  } else if (warp == 0) {
    // ============================================================ loads
    int kj = 0, vj = 0, qj = 0;
    bool ok = true;
    Unit u;
    const uint8_t* k4 = reinterpret_cast<const uint8_t*>(p.k_cache);
    const uint8_t* v4 = reinterpret_cast<const uint8_t*>(p.v_cache);
    while (ok && next_unit(u) && u.T >= 0) {
      const int qb = qj % C::NQ;
      if (qj >= C::NQ && !__all_sync(kAll, mbar_wait(bars.q_empty(qb), (qj / C::NQ - 1) & 1, abort_flag, kWaitNs))) break;
      if (lane == 0) {
        mbar_expect_tx(bars.q_full(qb), (uint32_t)p.rows_per_tile * 128u * (D / 64));
        for (int kb = 0; kb < D / 64; ++kb)
          tma_load_3d(smem_u32(sQ + qb * C::Q_BYTES + kb * (BN * 128)), &tm_q, bars.q_full(qb), kb * 64, u.g * p.G,
                      u.o0 + u.rt * p.rows_per_tile / p.G);
      }
      ++qj;
      const int64_t first_pos = WIN ? u.P - p.window + 1 : 0;
      // lane j < 8 looks after block j of a tile: its index, or -1 (not
      // loaded: past the end, or seen by no row), -2 (a bad page)
      auto block_of = [&](int t) -> int64_t {
        if (t >= u.npt || lane >= kBlocks) return -1;
        const int off = lane * kPageSize;
        if (t == u.npt - 1 && off >= u.tail) return -1;
        const int64_t v = u.k_begin + (int64_t)t * BK;
        const int64_t pos = (v < u.s0 ? v : v - u.s0 + u.w0) + off;
        if (WIN && pos >= p.sinks && pos + kPageSize <= first_pos) return -1;
        if (!p.paged) return ((int64_t)u.b * p.Hkv + u.g) * p.max_pages + pos / kPageSize;
        const int pid = p.page_table[(int64_t)u.b * p.max_pages + pos / kPageSize];
        return pid >= 0 && pid < p.num_pages ? (int64_t)pid * p.Hkv + u.g : -2;
      };
      auto load = [&](uint8_t* slot, uint32_t bar, const uint8_t* src, int bytes, int64_t blk) {
        if (blk == -2) {                                     // a bad page reads as zeros
          set_status(p.status, TV_DEV_BAD_PAGE);
          for (int o = 0; o < bytes; o += 16)
            *reinterpret_cast<uint4*>(slot + lane * bytes + o) = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
          fence_proxy_async_smem();
        }
        const int nb = __popc(__ballot_sync(kAll, blk >= 0));
        if (lane == 0) mbar_expect_tx(bar, (uint32_t)(nb * bytes));
        __syncwarp();
        if (blk >= 0) bulk_load(smem_u32(slot + lane * bytes), src + blk * bytes, (uint32_t)bytes, bar);
      };
      int64_t blk_k = -1, blk_v = -1, nx = block_of(0);
      for (int t = 0; t <= u.npt && ok; ++t) {
        blk_v = blk_k;
        blk_k = nx;
        nx = block_of(t + 1);
        if (t < u.npt) {
          const int i = kj % C::NK;
          if (kj >= C::NK && !__all_sync(kAll, mbar_wait(bars.k_empty(i), (kj / C::NK - 1) & 1, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          load(sK + i * C::K_SLOT, bars.k_full(i), k4, C::KB, blk_k);
          ++kj;
        }
        if (t >= 1) {
          const int i = vj % C::NV;
          if (vj >= C::NV && !__all_sync(kAll, mbar_wait(bars.v_empty(i), (vj / C::NV - 1) & 1, abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          load(sV + i * C::V_SLOT, bars.v_full(i), v4, C::VB, blk_v);
          ++vj;
        }
      }
    }
    // every copy this warp started has landed before the CTA exits
    if (lane == 0) {
      int spare = 0;
      for (int i = (qj > C::NQ ? qj - C::NQ : 0); i < qj; ++i) mbar_wait(bars.q_full(i % C::NQ), (i / C::NQ) & 1, &spare, kWaitNs);
      for (int i = (kj > C::NK ? kj - C::NK : 0); i < kj; ++i) mbar_wait(bars.k_full(i % C::NK), (i / C::NK) & 1, &spare, kWaitNs);
      for (int i = (vj > C::NV ? vj - C::NV : 0); i < vj; ++i) mbar_wait(bars.v_full(i % C::NV), (i / C::NV) & 1, &spare, kWaitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ MMA issue
    constexpr uint32_t ID_QK = idesc_bf16_f32(128, BN, 0, 0);
    constexpr uint32_t ID_PV = idesc_bf16_f32(128, BN, 0, 1);
    const uint32_t q_addr = smem_u32(sQ), p_addr = smem_u32(sP);
    int aj = 0, x = 0, unit = 0;                             // A operands, tiles, units so far
    bool ok = true;
    Unit u;
    while (ok && next_unit(u) && u.T >= 0) {
      if (lane == 0) {
        const int qb = unit % C::NQ, ob = unit % C::NO;
        ok = mbar_wait(bars.q_full(qb), (unit / C::NQ) & 1, abort_flag, kWaitNs);
        if (ok && unit >= C::NO) ok = mbar_wait(bars.o_empty(ob), (unit / C::NO - 1) & 1, abort_flag, kWaitNs);
        tc_fence_after();
        for (int t = 0; t <= u.T && ok; ++t) {
          if (t < u.T) {
            const int y = x + t, buf = y & 1;
            if (y >= 2 && !mbar_wait(bars.s_empty(buf), ((y - 2) >> 1) & 1, abort_flag, kWaitNs)) { ok = false; break; }
            for (int c = 0; c < C::CPT && ok; ++c, ++aj) {
              const int slot = aj % C::NA;
              if (!mbar_wait(bars.a_full(slot), (aj / C::NA) & 1, abort_flag, kWaitNs)) { ok = false; break; }
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const int kg = c * 8 + kk;                   // 16-channel step
                const uint64_t bd = smem_desc(q_addr + qb * C::Q_BYTES + (kg >> 2) * (BN * 128) + (kg & 3) * 32, 16, 1024, 2);
                mma_ts(tmem + C::T_S + buf * BN, tmem + C::T_A + slot * 64 + kk * 8, bd, ID_QK, (c > 0 || kk > 0) ? 1u : 0u);
              }
              mma_commit(bars.a_empty(slot));
            }
            if (!ok) break;
            mma_commit(bars.s_full(buf));
            if (t == u.T - 1) mma_commit(bars.q_empty(qb));
          }
          if (t >= 1) {
            const int y = x + t - 1, buf = y & 1;
            if (!mbar_wait(bars.p_full(buf), (y >> 1) & 1, abort_flag, kWaitNs)) { ok = false; break; }
            tc_fence_after();
            for (int c = 0; c < C::CPT && ok; ++c, ++aj) {
              const int slot = aj % C::NA;
              if (!mbar_wait(bars.a_full(slot), (aj / C::NA) & 1, abort_flag, kWaitNs)) { ok = false; break; }
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {               // 16-key step
                const uint64_t bd = smem_desc(p_addr + buf * P_BYTES + kk * (16 * 128), P_BYTES, 1024, 2);
                mma_ts(tmem + (ob * C::CPT + c) * BN, tmem + C::T_A + slot * 64 + kk * 8, bd, ID_PV, (t > 1 || kk > 0) ? 1u : 0u);
              }
              mma_commit(bars.a_empty(slot));
            }
            if (!ok) break;
            mma_commit(bars.pv_done(buf));
          }
        }
        x += u.T;
        ++unit;
      }
      ok = __shfl_sync(kAll, (int)ok, 0) != 0;
    }
    if (lane == 0) {
      // every MMA this thread issued has finished before tensor memory is freed
      int spare = 0;
      mma_commit(bars.fin());
      mbar_wait(bars.fin(), 0, &spare, kWaitNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + kExpandWarps) {
    // ============================================================ expansion
    const int grp = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const __nv_bfloat16* kt = reinterpret_cast<const __nv_bfloat16*>(p.k_tree);
    const __nv_bfloat16* vt = reinterpret_cast<const __nv_bfloat16*>(p.v_tree);
    int aj = 0, kj = 0, vj = 0;
    bool ok = true;
    Unit u;
    while (ok && next_unit(u) && u.T >= 0) {
      for (int t = 0; t <= u.T && ok; ++t)
        for (int kind = 0; kind < 2 && ok; ++kind) {         // 0: K(t), 1: V(t - 1)
          const int tile = t - kind;
          if (tile < 0 || tile >= u.T) continue;
          const bool tree = tile == u.npt;
          for (int c = 0; c < C::CPT && ok; ++c, ++aj) {
            if ((aj & 1) != grp) continue;
            const int slot = aj % C::NA;
            const uint32_t dst = tmem + lane_base + C::T_A + slot * 64;
            const int ring = kind == 0 ? kj % C::NK : vj % C::NV;
            if (!tree) {
              const bool in = kind == 0 ? mbar_wait(bars.k_full(ring), (kj / C::NK) & 1, abort_flag, kWaitNs)
                                        : mbar_wait(bars.v_full(ring), (vj / C::NV) & 1, abort_flag, kWaitNs);
              if (!__all_sync(kAll, in)) { ok = false; break; }
            }
            if (aj >= C::NA && !__all_sync(kAll, mbar_wait(bars.a_empty(slot), (aj / C::NA - 1) & 1, abort_flag, kWaitNs))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (!tree && kind == 0) {
              // lane = key: four groups of 32 channels, 16 bytes and a scale each
              const uint8_t* blk = sK + ring * C::K_SLOT + (row >> 4) * C::KB;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const int gr = 4 * c + 2 * h + q;
                  const uint4 w4 = *reinterpret_cast<const uint4*>(blk + kv4::k_code(gr, row & 15));
                  const uint32_t code = blk[kv4::k_scale(D, gr, row & 15)];
                  const uint32_t s2 = ((code << 4) + 0x3800u) * 0x00010001u;    // the scale as a bf16 pair
                  const uint32_t o2 = fma_bf16x2(s2, kMinus136, kZero);
                  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                  for (int e = 0; e < 16; ++e) r[16 * q + e] = fma_bf16x2(pair_of(w[e >> 2], e & 3), s2, o2);
                }
                tmem_st32(dst + 32 * h, r);
              }
            } else if (!tree) {
              // lane = channel: 8 bytes (16 keys) of each block
              const uint8_t* src = sV + ring * C::V_SLOT + kv4::v_code(c * 128 + row);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint2 w2 = *reinterpret_cast<const uint2*>(src + (4 * h + q) * C::VB);
#pragma unroll
                  for (int e = 0; e < 8; ++e) r[8 * q + e] = fma_bf16x2(pair_of(e < 4 ? w2.x : w2.y, e & 3), kOne, kMinus136);
                }
                tmem_st32(dst + 32 * h, r);
              }
            } else if (kind == 0) {
              // the tree's keys, rows of k_tree; rows past the tree are zeros
              const uint4* src = reinterpret_cast<const uint4*>(kt + ((int64_t)u.g * p.R + u.o0 + row) * D + c * 128);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint4 w = row < u.n ? __ldg(src + 8 * h + e) : make_uint4(0, 0, 0, 0);
                  r[4 * e] = w.x;
                  r[4 * e + 1] = w.y;
                  r[4 * e + 2] = w.z;
                  r[4 * e + 3] = w.w;
                }
                tmem_st32(dst + 32 * h, r);
              }
            } else {
              // the tree's values: channel `row` of every node, node pairs
              const uint16_t* src = reinterpret_cast<const uint16_t*>(vt) + ((int64_t)u.g * p.R + u.o0) * D + c * 128 + row;
              uint32_t r[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t lo = 2 * e < u.n ? __ldg(src + (int64_t)(2 * e) * D) : 0u;
                const uint32_t hi = 2 * e + 1 < u.n ? __ldg(src + (int64_t)(2 * e + 1) * D) : 0u;
                r[e] = lo | (hi << 16);
              }
              tmem_st32(dst, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = 0u;
              tmem_st32(dst + 32, r);
            }
            if (!tree) {                                     // the packed bytes are in registers
              __syncwarp();
              if (lane == 0) mbar_arrive(kind == 0 ? bars.k_empty(ring) : bars.v_empty(ring));
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.a_full(slot));
          }
          if (!tree) kind == 0 ? ++kj : ++vj;
        }
    }
  } else if (warp >= 4 + kExpandWarps) {
    // ============================================================ softmax
    Softmax<D, WIN> sm{p, bars, sh, sP, sV, tmem};
    Unit u;
    bool ok = true;
    while (ok) {
      // the group goes on or stops together: its barriers have no limit of their own
      const bool got = next_unit(u);
      if (group_or(1 + ((warp - 4 - kExpandWarps) >> 2), !got) || u.T < 0) break;
      const int live = min(p.rows_per_tile, u.n * p.G - u.rt * p.rows_per_tile);
      ok = live > 32 ? sm.template run<32>(u) : (live > 16 ? sm.template run<16>(u) : sm.template run<8>(u));
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(p.status, TV_DEV_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
    else
      cudaGetLastError();
  });
  return fn;
}

template <int D, bool WIN>
cudaError_t launch_t(const AttnParams& p, cudaStream_t st) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorInvalidValue;
  CUtensorMap mq;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.R};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * p.Hq};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(BN / p.G)}, es[3] = {1, 1, 1};
  if (fn(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cudaError_t e = ensure_max_dynamic_smem<tv_attn_kv4_kernel<D, WIN>>((int)Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.B * p.Hkv * p.row_tiles * p.splits;
  const int64_t sms = num_sms();
  return launch_dep(tv_attn_kv4_kernel<D, WIN>, dim3((unsigned)(units < sms ? units : sms)), dim3(kThreads),
                    Cfg<D>::SMEM, st, p, mq);
}

template <bool WIN>
cudaError_t launch_d(const AttnParams& p, cudaStream_t s) {
  if (p.d == 128) return launch_t<128, WIN>(p, s);
  if (p.d == 256) return launch_t<256, WIN>(p, s);
  return launch_t<512, WIN>(p, s);
}

}  // namespace

bool kv4_tc_supported(const tv_desc* d, int G) { return d->dtype == TV_BF16 && G <= BN; }

int kv4_tc_rows(int G) { return BN / G * G; }

int kv4_tc_key_tile() { return BK; }

cudaError_t launch_attn_kv4(const AttnParams& p, cudaStream_t s) {
  return p.window > 0 ? launch_d<true>(p, s) : launch_d<false>(p, s);
}

}  // namespace tv
