// tcgen05 split-KV tree-verify attention over a 4-bit cache (tree_kv4.h):
// bf16 queries and tree K/V, fp32 accumulation and softmax, head_dim 128, 256
// or 512.
//
// The method is flash-decode with a tree mask: a CTA (tile of query rows, KV
// head, chunk of keys, sequence) leaves a normalised partial output with its
// reference exponent m and its sum l, and the log-sum-exp merge joins the
// chunks.
//
// Both products are taken transposed, so that the cache's values are the A
// operand and go from registers into tensor memory, never through shared
// memory, and so that N = 16 .. 128 query rows cost N columns:
//   S^T [128 keys x N rows]     = K  [keys x d]        Q^T   (A: tensor memory, B: Q in shared memory)
//   O^T [128 channels x N rows] += V^T [channels x keys] P^T  (A: tensor memory, B: P in shared memory)
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
// Every compute warp does every step of a tile: expand K (a tile ahead where
// tensor memory has room for two score tiles), softmax, expand V; one warp
// issues the MMAs and one copies the packed blocks ahead into a ring.  4, 2 or
// 1 such CTAs share an SM (128, 256 or 512 columns of tensor memory), so that
// one's products and waits run beside another's arithmetic.  A first build with
// a warp group per step and a persistent CTA per SM was bound by its hand-offs
// and by instruction fetch over five kinds of loops (64 sequences x 1 row over
// up to 16384 keys: 422 us against 264 us).
//
// Measured: a tree of 60 nodes x 4 heads over 32768 keys (head_dim 256) 51 us,
// 630 TFLOP/s; 16 ragged trees over up to 8192 keys (128, paged) 164 us, 310
// TFLOP/s.  What bounds it is the compute warps' work and the chain of its
// steps: expansion (2.75 instructions a pair of values, for each tile of query
// rows again), exponents, two barriers a tile; 47% of the issue slots at one
// CTA of 128 columns an SM.  Narrower tiles expand more often: 64 columns took
// 78 and 229 us where 128 took 56 and 190 (the same two calls, an earlier
// build).
//
// Every mbarrier wait is bounded (1 s); on a timeout the CTA raises
// TV_DEV_TIMEOUT, waits for its own copies and MMAs, frees tensor memory and
// returns.
#include <cuda.h>

#include <climits>
#include <type_traits>

#include "tc_ptx.cuh"
#include "tv_kv4.cuh"
#include "tv_tensormap.cuh"

namespace tv {
namespace {

using namespace tc;
using kv4::fma_bf16x2;
using kv4::kMinus136;
using kv4::kMinusZero;
using kv4::kOne;
using kv4::PairBits;

constexpr int BK = 128;                          // keys per tile
constexpr int kBlocks = BK / kPageSize;          // cache blocks per tile
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kHeadroom = 60.0f;               // log2: a weight above 2^60 moves the reference
constexpr uint32_t kHeader = 6144;

// head_dim D, N query rows per tile
template <int D, int N>
struct Cfg {
  static constexpr int CPT = D / 128;                       // 128-channel chunks of a tile
  static constexpr int KB = kv4::k_block_bytes(D), VB = kv4::v_block_bytes(D);
  // tensor memory columns: scores (two tiles where they fit), outputs, A operands of 64 columns
  static constexpr int USED = N + CPT * N + 64;
  static constexpr int TCOLS = USED <= 128 && N < 32 ? 128 : (USED <= 256 ? 256 : 512);
  static constexpr bool PIPE = TCOLS >= 2 * N + CPT * N + 64;
  static_assert(PIPE || CPT > 1, "the V slot is read (scales) after its first chunk is expanded");
  static constexpr int T_S = 0, T_O = N * (PIPE ? 2 : 1), T_A = T_O + CPT * N;
  static constexpr int NS = TCOLS - T_A >= 128 ? 2 : 1;     // A operands
  // one chunk and an operand each for K and V: V is expanded before the softmax, so that its product can start at once
  static constexpr bool V_FIRST = PIPE && CPT == 1 && NS == 2;
  static constexpr int CTAS = 512 / TCOLS;                  // per SM
  static constexpr int GPT = TCOLS / 128;                   // warp groups of 128 lanes
  static constexpr int HC = N / GPT < 16 ? 16 : N / GPT;    // rows per softmax thread
  static constexpr int kWarps = 4 * GPT, kCompute = 32 * kWarps, kThreads = kCompute + 64;
  // ring slots that the shared memory of CTAS CTAs per SM holds
  static constexpr int NK = D == 128 ? (N == 128 ? 6 : (N == 64 ? 4 : (N == 32 ? 4 : 2)))
                                     : (D == 256 ? (N == 16 ? 1 : 2) : (N == 64 ? 2 : 1));
  static constexpr int NV = D == 256 && N == 64 ? 1 : NK;
  static constexpr int P_COLS = N < 64 ? N : 64;            // columns of a P box: rows of 32, 64 or 128 bytes
  static constexpr uint32_t P_PITCH = 2 * P_COLS, P_BOX = BK * P_PITCH, P_BYTES = BK * 2 * N;
  static constexpr uint32_t P_SWIZZLE = P_COLS == 64 ? 2 : (P_COLS == 32 ? 4 : 6);
  static constexpr uint32_t Q_BYTES = N * D * 2;
  static constexpr uint32_t K_SLOT = kBlocks * KB, V_SLOT = kBlocks * VB;
  static constexpr uint32_t SMEM = kHeader + Q_BYTES + P_BYTES + NK * K_SLOT + NV * V_SLOT;
  static_assert(T_A + NS * 64 <= TCOLS, "tensor memory");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024 && SMEM <= 232448, "shared memory");
  // barriers: ring slots, A operands written and multiplied, scores done, products done, queries, end
  static constexpr int kKFull = 0, kKEmpty = NK, kVFull = 2 * NK, kVEmpty = 2 * NK + NV, kAFull = 2 * (NK + NV),
                       kADone = kAFull + NS, kS = kADone + NS, kPV = kS + 2, kQ = kPV + 1, kFin = kQ + 1, kBars = kFin + 1;
  static_assert(kBars * 8 <= 512, "barriers overflow their area");
};

__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};\n"
      :
      : "r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Eight k-steps D (+)= A[tmem] x B[smem] as one block: the operands advance by
// constants (A 8 columns a step, B S1 sixteen-byte units, from the fifth step
// on S4 - 4 S1 more), so that issuing costs few instructions beside the MMAs.
template <uint32_t S1, uint32_t S4>
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      ".reg .b32 a<8>;\n"
      ".reg .b64 b<8>;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n add.u32 a4, %1, 32;\n"
      "add.u32 a5, %1, 40;\n add.u32 a6, %1, 48;\n add.u32 a7, %1, 56;\n"
      "add.u64 b1, %2, %5;\n add.u64 b2, %2, 2 * %5;\n add.u64 b3, %2, 3 * %5;\n add.u64 b4, %2, %6;\n"
      "add.u64 b5, %2, %6 + %5;\n add.u64 b6, %2, %6 + 2 * %5;\n add.u64 b7, %2, %6 + 3 * %5;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, 1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, 1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, 1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b4, %3, 1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b5, %3, 1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b6, %3, 1;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b7, %3, 1;\n"
      "}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(S1), "n"(S4)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }


__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[16]) { tmem_ld_x16(a, r); }
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&r)[32]) { tmem_ld_x32(a, r); }

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

// Barrier of THREADS threads with the OR of a predicate over them: id 1, the
// compute warps; id 2, they and the MMA warp.
template <int ID, int THREADS>
__device__ __forceinline__ bool bar_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "bar.red.or.pred q, %2, %3, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(ID), "n"(THREADS)
      : "memory");
  return r != 0;
}

// 16 bytes global -> shared; cp_async_arrive: an arrival on an mbarrier when
// the thread's copies so far have landed
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(v) : "memory");
}

// pairs of fp32 numbers in one operation
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
  alignas(16) float nm[128];                     // -reference of each row (-inf: not a row)
  float red[16][32];                             // per-warp column results
  alignas(16) float inv[128];
  uint64_t anc[128];
  int dep[128];
  uint32_t none[4];                              // rows of a group without a reference yet
  uint32_t tmem;
  int abort_flag;
};
static_assert(512 + sizeof(Shared) <= kHeader, "header");

// mbar_sleep_wait with the polling loop out of line: the many waits would
// otherwise fill the instruction cache
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_sleep_wait(bar, parity, abort_flag, kWaitNs);
}
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait_hint(bar, parity) || wait_long(bar, parity, abort_flag);
}

template <int D, int N, bool WIN>
__global__ void __launch_bounds__(Cfg<D, N>::kThreads, Cfg<D, N>::CTAS)
tv_attn_kv4_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap tm_q) {
  using C = Cfg<D, N>;
  constexpr int CPT = C::CPT, NS = C::NS, HC = C::HC;
  constexpr unsigned kAll = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw + 512);
  uint8_t* sQ = smem_raw + kHeader;
  uint8_t* sP = sQ + C::Q_BYTES;
  uint8_t* sK = sP + C::P_BYTES;
  uint8_t* sV = sK + C::NK * C::K_SLOT;
  const uint32_t bars = smem_u32(smem_raw);
  auto bar = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };
  volatile int* abort_flag = &sh.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // the swizzled tiles need the dynamic shared window to start 1 KB aligned
  if (smem_u32(smem_raw) & 1023u) {
    dep_wait();
    if (tid == 0) set_status(p.status, TV_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::kBars; ++i) {
      const bool by_warp = i >= C::kAFull && i < C::kADone;
      const bool by_lane = i < C::kKEmpty || (i >= C::kVFull && i < C::kVEmpty);
      mbar_init(bar(i), by_lane ? 32 : (by_warp ? C::kWarps : 1));   // the copying lanes, the compute warps, or one
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (p.rows_per_tile < N) {
    // pad rows of the query tile (G does not divide N) hold zeros
    const int pad = N - p.rows_per_tile;
    for (int e = tid; e < (D / 64) * pad * 8; e += C::kThreads) {
      const int kb = e / (pad * 8), r = p.rows_per_tile + (e / 8) % pad, c = e % 8;
      *reinterpret_cast<uint4*>(sQ + kb * (N * 128) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sh.tmem), C::TCOLS);
    tmem_relinquish();
  }
  if (tid == C::kCompute + 32) tma_prefetch_desc(&tm_q);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  dep_wait();
  dep_launch();

  // ---------------------------------------------------------------- work
  const int rt = blockIdx.x, g = blockIdx.y / p.splits, s_id = blockIdx.y % p.splits, b = blockIdx.z;
  const int64_t Praw = p.prefix_len[b];            // read together with the offsets
  int o0 = 0, n = 1;
  bool active = seq_rows(p.node_offsets, b, p.R, p.max_nodes, p.status, &o0, &n);
  const int m0 = rt * p.rows_per_tile, nlive = min(p.rows_per_tile, n * p.G - m0);
  active = active && nlive > 0;
  const int64_t P = clamp_prefix(Praw, p.max_prefix, p.capacity);
  if (active && P != Praw && tid == 0 && rt == 0 && s_id == 0 && g == 0) set_status(p.status, TV_DEV_BAD_PREFIX);
  const KeyMap km = key_map(P, WIN ? p.window : 0, p.sinks, p.map_tile);
  const int nch = num_chunks(km.len, p.chunk, p.tree_tile);
  active = active && s_id < nch;                   // uniform over the CTA
  const int64_t k_begin = (int64_t)s_id * p.chunk, k_end = min(km.len, k_begin + p.chunk);
  const int npt = k_end > k_begin ? (int)((k_end - k_begin + BK - 1) / BK) : 0;   // prefix tiles
  const int T = npt + (s_id == nch - 1 ? 1 : 0);
  const int tail = npt > 0 ? (int)(k_end - k_begin - (int64_t)(npt - 1) * BK) : BK;
  const int64_t first_pos = WIN ? P - p.window + 1 : 0;      // positions [sinks, first_pos) are seen by no row
  auto tile_pos = [&](int t) -> int64_t {
    const int64_t v = k_begin + (int64_t)t * BK;
    return WIN ? km.pos(v) : v;
  };

  if (!active) {
    // nothing to do for this CTA: straight to teardown
  } else if (warp == C::kWarps + 1) {
    // ============================================================ loads
    if (lane == 0) {
      mbar_expect_tx(bar(C::kQ), (uint32_t)p.rows_per_tile * 128u * (D / 64));
      for (int kb = 0; kb < D / 64; ++kb)
        tma_load_3d(smem_u32(sQ + kb * (N * 128)), &tm_q, bar(C::kQ), kb * 64, g * p.G, o0 + m0 / p.G);
    }
    const uint8_t* k4 = reinterpret_cast<const uint8_t*>(p.k_cache);
    const uint8_t* v4 = reinterpret_cast<const uint8_t*>(p.v_cache);
    // Four lanes copy one block, 16 bytes a lane and instruction, addresses at
    // constant offsets: a bulk copy per block cost more instructions (one
    // lane's operands at a time) than the copies of all lanes together.
    const int blk_of_lane = lane >> 2;
    // at(t): number of the lane's block of tile t in its sequence, -1 where
    // nothing is loaded (past the end, or seen by no row); ids(t): what the page
    // table holds for it (any number), read two tiles before its use
    auto at = [&](int t) -> int64_t {
      const int off = blk_of_lane * kPageSize;
      if (t >= npt || (t == npt - 1 && off >= tail)) return -1;
      const int64_t pos = tile_pos(t) + off;
      return WIN && pos >= p.sinks && pos + kPageSize <= first_pos ? -1 : pos / kPageSize;
    };
    auto ids = [&](int t) -> int {
      const int64_t i = p.paged ? at(t) : -1;
      return i < 0 ? 0 : p.page_table[(int64_t)b * p.max_pages + i];
    };
    const uint32_t k_dst = smem_u32(sK) + blk_of_lane * C::KB + (lane & 3) * 16;
    const uint32_t v_dst = smem_u32(sV) + blk_of_lane * C::VB + (lane & 3) * 16;
    // BYTES of a block, starting at the lane's 16
    auto copy = [&](uint32_t dst, const uint8_t* src, auto bytes) {
      constexpr int kChunks = decltype(bytes)::value / 16;
#pragma unroll 17
      for (int i = 0; i < kChunks / 4; ++i) cp_async16(dst + i * 64, src + i * 64);
      if (kChunks % 4 > (lane & 3)) cp_async16(dst + kChunks / 4 * 64, src + kChunks / 4 * 64);
    };
    int id0 = ids(0), id1 = ids(1), ks = 0, vs = 0, kp = 1, vp = 1;
    bool ok = true;
    for (int t = 0; t < npt; ++t) {
      const int raw = id0;
      id0 = id1;
      id1 = ids(t + 2);
      int64_t blk = at(t);
      if (blk >= 0) {
        if (!p.paged)
          blk += ((int64_t)b * p.Hkv + g) * p.max_pages;
        else
          blk = raw >= 0 && raw < p.num_pages ? (int64_t)raw * p.Hkv + g : -2;
      }
      // a bad page is flagged and reads as zeros
      if (blk == -2) set_status(p.status, TV_DEV_BAD_PAGE);
      auto put = [&](uint32_t dst, const uint8_t* src, auto bytes, uint32_t full) {
        if (blk >= 0) {
          copy(dst, src + blk * decltype(bytes)::value + (lane & 3) * 16, bytes);
          cp_async_arrive(full);
          return;
        }
        if (blk == -2)
          for (uint32_t o = 0; o + (lane & 3) * 16 < (uint32_t)decltype(bytes)::value; o += 64) st_shared16(dst + o, 0x88888888u);
        mbar_arrive(full);
      };
      // (K of this tile never waits for V of the one before: the compute warps take it first)
      if (t >= C::NK) ok = wait_on(bar(C::kKEmpty + ks), kp, abort_flag);
      if (!__all_sync(kAll, ok)) break;
      put(k_dst + ks * C::K_SLOT, k4, std::integral_constant<int, C::KB>(), bar(C::kKFull + ks));
      if (t >= C::NV) ok = wait_on(bar(C::kVEmpty + vs), vp, abort_flag);
      if (!__all_sync(kAll, ok)) break;
      put(v_dst + vs * C::V_SLOT, v4, std::integral_constant<int, C::VB>(), bar(C::kVFull + vs));
      if (++ks == C::NK) {
        ks = 0;
        kp ^= 1;
      }
      if (++vs == C::NV) {
        vs = 0;
        vp ^= 1;
      }
    }
    // every copy this warp started has landed before the CTA exits
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
      int spare = 0;
      wait_on(bar(C::kQ), 0, &spare);
    }
    __syncwarp();
  } else if (warp == C::kWarps) {
    // ============================================================ MMA issue
    constexpr uint32_t ID_QK = idesc_bf16_f32(128, N, 0, 0), ID_PV = idesc_bf16_f32(128, N, 0, 1);
    const uint64_t q_desc = smem_desc(smem_u32(sQ), 16, 1024, 2);
    const uint64_t p_desc = smem_desc(smem_u32(sP), C::P_BOX, 8 * C::P_PITCH, C::P_SWIZZLE);
    bool ok = __all_sync(kAll, wait_on(bar(C::kQ), 0, abort_flag));
    uint32_t slot = 0, par = 0;                              // next A operand and its phase
    int ks = 0, vs = 0;                                      // ring slots: free once every compute warp has expanded them
    auto operand = [&]() {
      ok = __all_sync(kAll, wait_on(bar(C::kAFull + slot), par, abort_flag)) && ok;
      tc_fence_after();
    };
    auto advance = [&]() {
      if (++slot == NS) {
        slot = 0;
        par ^= 1;
      }
    };
    auto scores_of = [&](int t) {
      const uint32_t buf = C::PIPE ? (uint32_t)t & 1u : 0u;
#pragma unroll 1
      for (int c = 0; c < CPT; ++c) {
        operand();
        if (elect_one()) {
          mma8_ts<2, N * 8>(tmem + C::T_S + buf * N, tmem + C::T_A + slot * 64, q_desc + (uint32_t)c * (2 * N * 8), ID_QK,
                            c > 0 ? 1u : 0u);
          mma_commit(bar(C::kADone + slot));
          if (c == CPT - 1) {
            mma_commit(bar(C::kS + buf));
            if (t != npt) mbar_arrive(bar(C::kKEmpty + ks));
          }
        }
        __syncwarp();
        advance();
      }
      if (++ks == C::NK) ks = 0;
    };
    scores_of(0);
    for (int t = 0; t < T; ++t) {
      if (C::PIPE && t + 1 < T) scores_of(t + 1);
      if (bar_or<2, C::kCompute + 32>(!ok)) {                // the tile's weights are in P, or (rare) need another pass
        if (bar_or<2, C::kCompute + 32>(!ok)) break;
        bar_or<2, C::kCompute + 32>(false);
      }
#pragma unroll 1
      for (int c = 0; c < CPT; ++c) {
        operand();
        if (elect_one()) {
          mma8_ts<C::P_PITCH, 4 * C::P_PITCH>(tmem + C::T_O + c * N, tmem + C::T_A + slot * 64, p_desc, ID_PV, t > 0 ? 1u : 0u);
          mma_commit(bar(C::kADone + slot));
          if (c == CPT - 1) {
            mma_commit(bar(C::kPV));
            if (t != npt) mbar_arrive(bar(C::kVEmpty + vs));
          }
        }
        __syncwarp();
        advance();
      }
      if (++vs == C::NV) vs = 0;
      if (!C::PIPE && t + 1 < T) scores_of(t + 1);
    }
    if (elect_one()) {
      // every MMA this thread issued has finished before tensor memory is freed
      int spare = 0;
      mma_commit(bar(C::kFin));
      wait_on(bar(C::kFin), 0, &spare);
    }
    __syncwarp();
  } else {
    // ============================================================ compute
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane;       // row: TMEM lane (key of K, channel of V)
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t a_base = tmem + lane_base + C::T_A;
    const float c2 = p.scale_log2;
    const int c0 = grp * HC, live = max(0, min(HC, nlive - c0));   // this group's softmax columns
    float* nm = sh.nm + c0;

    if (c0 < N && row < HC) {
      const int m = m0 + c0 + row;
      const bool ok = row < live;
      if (T > npt || WIN) {
        sh.anc[c0 + row] = ok ? p.anc[o0 + m / p.G] : 0ull;
        if (WIN) sh.dep[c0 + row] = ok ? p.depth[o0 + m / p.G] : 0;
      }
      nm[row] = ok ? 0.f : -INFINITY;
    }
    if (row == 0) sh.none[grp] = live == 32 ? 0xffffffffu : (1u << live) - 1u;
    uint64_t l2[HC / 2];
#pragma unroll
    for (int j = 0; j < HC / 2; ++j) l2[j] = 0ull;

    const PairBits pair;
    constexpr int H = 4 / C::GPT;                                  // 16-column pieces of an A operand per group
    // this lane's bytes of a ring slot: K, row = key; V, row = channel
    const uint8_t* k_lane = sK + (row >> 4) * C::KB + kv4::k_code(grp * H, row & 15);
    const uint8_t* k_scale_lane = sK + (row >> 4) * C::KB + kv4::k_scale(D, grp * H, row & 15);
    const uint8_t* v_lane = sV + kv4::v_code(row) + 2 * grp * H * C::VB;
    const uint8_t* v_scale_lane = sV + (row >> 4) * C::VB + kv4::v_scale(D, row & 15);
    uint8_t* prow = sP + (c0 / C::P_COLS) * C::P_BOX + row * C::P_PITCH;
    const uint32_t swz = C::P_COLS == 64 ? (uint32_t)(row & 7) : (C::P_COLS == 32 ? (uint32_t)(row >> 1) & 3u : (uint32_t)(row >> 2) & 1u);

    int ks = 0, vs = 0, kp = 0, vp = 0;
    uint32_t slot = 0, par = 1;                                    // next A operand; the phase of its use before
    bool bad = false, good = true;                                 // a wait gave up; all warps went on
    auto wait = [&](int i, uint32_t parity) {
      if (__builtin_expect(!mbar_try_wait_hint(bar(i), parity), 0)) bad |= !wait_long(bar(i), parity, abort_flag);
    };
    auto slot_written = [&]() {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kAFull + slot));
      if (++slot == NS) {
        slot = 0;
        par ^= 1;
      }
    };
    // Before an A operand is written, the MMAs that read it last (NS operands
    // before) are done.  Ahead of the scores (PIPE), K's first NS chunks follow
    // V of two tiles back, or K of the tile before, whose products the loop has
    // waited for; so does V where it goes first.
    auto expand_k = [&](int t) {
      const bool tree = t == npt;
      if (!tree) wait(C::kKFull + ks, kp);
#pragma unroll 1
      for (int c = 0; c < CPT; ++c) {
        if (c >= NS || (!C::PIPE && t > 0)) wait(C::kADone + slot, par);
        __syncwarp();
        tc_fence_after();
        const uint32_t dst = a_base + slot * 64 + grp * H * 16;
        if (!tree) {
          // lane = key: groups of 32 channels, 16 bytes and a scale each
          const uint8_t* code = k_lane + ks * C::K_SLOT + c * 1024;
          const uint8_t* scale = k_scale_lane + ks * C::K_SLOT + c * 64;
#pragma unroll 1
          for (int h = 0; h < H; ++h) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(code + h * 256);
            const uint32_t s2 = (((uint32_t)scale[h * 16] << 4) + 0x3800u) * 0x00010001u;   // the scale as a bf16 pair
            const uint32_t o2 = fma_bf16x2(s2, kMinus136, kMinusZero);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = fma_bf16x2(pair(w[e >> 2], e & 3), s2, o2);
            tmem_st16(dst + 16 * h, r);
          }
        } else {
          // the tree's keys, rows of k_tree; rows past the tree are zeros
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.k_tree) +
                                                            ((int64_t)g * p.R + o0 + row) * D + c * 128) + 4 * grp * H;
#pragma unroll 1
          for (int h = 0; h < H; ++h) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 w = row < n ? __ldg(src + 4 * h + e) : make_uint4(0, 0, 0, 0);
              r[4 * e] = w.x;
              r[4 * e + 1] = w.y;
              r[4 * e + 2] = w.z;
              r[4 * e + 3] = w.w;
            }
            tmem_st16(dst + 16 * h, r);
          }
        }
        slot_written();
      }
      if (!tree && ++ks == C::NK) {
        ks = 0;
        kp ^= 1;
      }
    };
    auto expand_v = [&](int t, int c) {
      const bool tree = t == npt;
      if ((!C::PIPE || C::V_FIRST) && !tree && c == 0) wait(C::kVFull + vs, vp);
      if (!C::V_FIRST) wait(C::kADone + slot, par);
      __syncwarp();
      tc_fence_after();
      const uint32_t dst = a_base + slot * 64 + grp * H * 16;
      if (!tree) {
        // lane = channel: 8 bytes (16 keys) of each block
        const uint8_t* src = v_lane + vs * C::V_SLOT + c * 1024;
#pragma unroll 1
        for (int h = 0; h < H; ++h) {
          const uint2 x = *reinterpret_cast<const uint2*>(src + (2 * h) * C::VB);
          const uint2 y = *reinterpret_cast<const uint2*>(src + (2 * h + 1) * C::VB);
          const uint32_t w[4] = {x.x, x.y, y.x, y.y};
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = fma_bf16x2(pair(w[e >> 2], e & 3), kOne, kMinus136);
          tmem_st16(dst + 16 * h, r);
        }
      } else {
        // the tree's values: channel `row` of every node, node pairs; zeros past the tree
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.v_tree) + ((int64_t)g * p.R + o0) * D + c * 128 + row;
#pragma unroll 1
        for (int h = 0; h < H; ++h) {
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int node = 32 * (grp * H + h) + 2 * e;
            const uint32_t lo = node < n ? __ldg(src + (int64_t)node * D) : 0u;
            const uint32_t hi = node + 1 < n ? __ldg(src + (int64_t)(node + 1) * D) : 0u;
            r[e] = lo | (hi << 16);
          }
          tmem_st16(dst + 16 * h, r);
        }
      }
      slot_written();
    };

    expand_k(0);
    for (int t = 0; t < T; ++t) {
      const bool tree = t == npt;
      const uint32_t buf = C::PIPE ? (uint32_t)t & 1u : 0u;
      if (C::PIPE) {
        wait(C::kS + buf, (t >> 1) & 1);
        if (C::V_FIRST && t + 1 < T) expand_k(t + 1);
        if (t > 0) wait(C::kPV, (t - 1) & 1);                      // P is free, O holds the tiles before
        if (!C::V_FIRST && t + 1 < T) expand_k(t + 1);
        if (C::V_FIRST) expand_v(t, 0);
      } else {
        expand_v(t, 0);                                            // beside the scores' product
        wait(C::kS, t & 1);
        if (t > 0) wait(C::kPV, (t - 1) & 1);
      }
      // ---- the softmax of the tile
      float sv = 1.f;                                              // V scale of the thread's key
      if (!tree) {
        if (C::PIPE && !C::V_FIRST) wait(C::kVFull + vs, vp);
        sv = kv4::scale_of(v_scale_lane[vs * C::V_SLOT]);
      }
      __syncwarp();
      tc_fence_after();
      float s[HC];
      auto scores = [&]() {                                        // the masked scores, from tensor memory
        {
          uint32_t r[HC];
          ld_cols(tmem + lane_base + C::T_S + buf * N + c0, r);
#pragma unroll
          for (int j = 0; j < HC; ++j) s[j] = __uint_as_float(r[j]);
        }
        if (__builtin_expect(tree, 0)) {
          // the key's bit of each row's ancestors; with a window also rows
          // less than a window deeper than it
          const uint32_t* word = reinterpret_cast<const uint32_t*>(sh.anc + c0) + ((row >> 5) & 1);
          const uint32_t bit = row < kMaxNodes ? 1u << (row & 31) : 0u;
          int lim = INT_MAX;
          if (WIN && row < n) {
            const int kd = p.depth[o0 + row];
            if (P + kd >= p.sinks) lim = (int)min((int64_t)INT_MAX, kd + p.window);
          }
#pragma unroll
          for (int j = 0; j < HC; ++j) {
            bool vis = (word[2 * j] & bit) != 0;
            if (WIN) vis = vis && sh.dep[c0 + j] < lim;
            if (!vis) s[j] = -INFINITY;
          }
          return;
        }
        if (WIN) {
          const int64_t p0 = tile_pos(t), pos = p0 + row;
          if (p0 < P + kMaxNodes - p.window) {
            // rows at most this deep see the key
            const int lim = pos < p.sinks ? INT_MAX : (int)max((int64_t)-1, min((int64_t)INT_MAX, pos - first_pos));
#pragma unroll
            for (int j = 0; j < HC; ++j)
              if (sh.dep[c0 + j] > lim) s[j] = -INFINITY;
          }
        }
        if (__builtin_expect(t == npt - 1 && row >= tail, 0)) {
#pragma unroll
          for (int j = 0; j < HC; ++j) s[j] = -INFINITY;
        }
      };
      const bool mine = live > 0;
      if (mine) scores();
      const bool by_row = tree || (WIN && tile_pos(t) < P + kMaxNodes - p.window);
      if (__builtin_expect(t == 0 && !by_row, 0)) {
        // every row sees key 0: its scores are the references
        if (row == 0 && mine) {
#pragma unroll
          for (int j = 0; j < HC; ++j)
            if (j < live) nm[j] = -s[j] * c2;
          sh.none[grp] = 0;
        }
        bar_or<1, C::kCompute>(false);
      }
      // weights into the P tile and, kept for the sums, in s
      auto weights = [&]() -> float {
        float xm = -INFINITY;
        const uint64_t cc = pack2(c2, c2), vv = pack2(sv, sv);
#pragma unroll
        for (int j8 = 0; j8 < HC / 8; ++j8) {
          const ulonglong2 na = reinterpret_cast<const ulonglong2*>(nm)[2 * j8], nb = reinterpret_cast<const ulonglong2*>(nm)[2 * j8 + 1];
          const uint64_t nn[4] = {na.x, na.y, nb.x, nb.y};
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& x = s[8 * j8 + 2 * e];
            float& y = s[8 * j8 + 2 * e + 1];
            unpack2(fma2(pack2(x, y), cc, nn[e]), x, y);
            xm = fmaxf(fmaxf(xm, x), y);
            x = ex2(x);
            y = ex2(y);
            float a, b2;
            unpack2(mul2(pack2(x, y), vv), a, b2);
            w[e] = pack_bf16(a, b2);
          }
          *reinterpret_cast<uint4*>(prow + (((uint32_t)((c0 % C::P_COLS) / 8 + j8) ^ swz) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return xm;
      };
      float xm = -INFINITY;
      if (mine) xm = weights();
      fence_proxy_async_smem();
      tc_fence_before();
      if (__builtin_expect(bar_or<2, C::kCompute + 32>(bad || xm > kHeadroom || (mine && sh.none[grp] != 0)), 0)) {
        // a wait gave up, a score is far above its reference, or a row has
        // none yet: move the references to the columns' maxima (O holds the
        // finished products of every earlier tile) and start again
        if (bar_or<2, C::kCompute + 32>(bad)) {
          good = false;
          break;
        }
        tc_fence_after();
        if (mine) {
          scores();
#pragma unroll
          for (int j = 0; j < HC; ++j) s[j] = fmaf(s[j], c2, nm[j]);
          const float top = reduce_columns<MaxOp>(s);
          if (lane < HC) sh.red[warp][lane] = top;
        }
        const uint32_t none = sh.none[grp];
        bar_or<1, C::kCompute>(false);
        if (mine) {
          const int j0 = lane & (HC - 1);
          const bool fresh = (none >> j0) & 1u;                    // no reference, weights or sum yet
          const float mx = fmaxf(fmaxf(sh.red[4 * grp][j0], sh.red[4 * grp + 1][j0]),
                                 fmaxf(sh.red[4 * grp + 2][j0], sh.red[4 * grp + 3][j0]));
          const bool moves = lane < live && mx != -INFINITY && (fresh || mx > 0.f);
          const float d = moves ? mx : 0.f, alpha = moves && !fresh ? ex2(-d) : 1.f;
          const uint32_t found = __ballot_sync(kAll, lane < live && mx != -INFINITY);
#pragma unroll
          for (int j = 0; j < HC / 2; ++j)
            l2[j] = mul2(l2[j], pack2(__shfl_sync(kAll, alpha, 2 * j), __shfl_sync(kAll, alpha, 2 * j + 1)));
          if (t > 0 && __any_sync(kAll, alpha != 1.f)) {
#pragma unroll 1
            for (int q = 0; q < CPT * (HC / 8); ++q) {
              const int cc = q / (HC / 8), j8 = q % (HC / 8) * 8;
              const uint32_t at = tmem + lane_base + C::T_O + cc * N + c0 + j8;
              uint32_t r[8];
              tmem_ld_x8(at, r);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                r[j] = __float_as_uint(__uint_as_float(r[j]) * __shfl_sync(kAll, alpha, j8 + j));
              tmem_st_x8(at, r);
            }
          }
          if ((warp & 3) == 0) {
            if (lane < HC) nm[lane] -= d;
            if (lane == 0) sh.none[grp] = none & ~found;
          }
        }
        bar_or<1, C::kCompute>(false);
        if (mine) {
          scores();
          weights();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        bar_or<2, C::kCompute + 32>(false);
      }
#pragma unroll
      for (int j = 0; j < HC / 2; ++j) l2[j] = add2(l2[j], pack2(s[2 * j], s[2 * j + 1]));
      // ---- V^T, 128 channels at a time
#pragma unroll 1
      for (int c = C::PIPE && !C::V_FIRST ? 0 : 1; c < CPT; ++c) expand_v(t, c);
      if (!tree && ++vs == C::NV) {
        vs = 0;
        vp ^= 1;
      }
      if (!C::PIPE && t + 1 < T) expand_k(t + 1);
    }

    // ---- epilogue: the sums over the keys, then the rows of O / l
    if (good) {
      wait(C::kPV, (T - 1) & 1);
      __syncwarp();
      tc_fence_after();
      float l[HC];
#pragma unroll
      for (int j = 0; j < HC / 2; ++j) unpack2(l2[j], l[2 * j], l[2 * j + 1]);
      const float sum = reduce_columns<SumOp>(l);
      if (lane < HC) sh.red[warp][lane] = sum;
      good = !bar_or<1, C::kCompute>(bad);
    }
    if (good) {
      const bool direct = p.out != nullptr && nch == 1;
      const int64_t slot0 = partial_slot(s_id, b, g, rt, c0, p.Hkv, p.row_tiles, p.tile_stride, p.splits);
      if (row < live) {
        const float L = (sh.red[4 * grp][row] + sh.red[4 * grp + 1][row]) + (sh.red[4 * grp + 2][row] + sh.red[4 * grp + 3][row]);
        sh.inv[c0 + row] = L > 0.f ? 1.f / L : 0.f;
        if (!direct)
          p.ml_part[slot0 + (int64_t)row * p.splits] = make_float2(((sh.none[grp] >> row) & 1u) ? -INFINITY : -nm[row], L);
      }
      bar_or<1, C::kCompute>(false);
      // TMEM lane = channel of the chunk: a warp stores 128 bytes of a row at a time
      const float4* inv4 = reinterpret_cast<const float4*>(sh.inv + c0);
#pragma unroll 1
      for (int c = 0; c < CPT && live > 0; ++c) {
        uint32_t r[HC];
        ld_cols(tmem + lane_base + C::T_O + c * N + c0, r);
        const int ch = c * 128 + row;
        if (!direct) {
          float* dst = p.o_part + slot0 * D + ch;
          const int64_t step = (int64_t)p.splits * D;
#pragma unroll
          for (int j = 0; j < HC; j += 4) {
            const float4 w = inv4[j / 4];
            const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (j + e < live) *dst = __uint_as_float(r[j + e]) * f[e];
              dst += step;
            }
          }
        } else {
          int node = (m0 + c0) / p.G, head = (m0 + c0) % p.G;
#pragma unroll
          for (int j = 0; j < HC; ++j) {
            if (j < live) {
              const int64_t e = ((int64_t)(o0 + node) * p.Hq + g * p.G + head) * D + ch;
              const float v = __uint_as_float(r[j]) * sh.inv[c0 + j];
              if (p.out_bf16)
                reinterpret_cast<__nv_bfloat16*>(p.out)[e] = __float2bfloat16_rn(v);
              else
                reinterpret_cast<float*>(p.out)[e] = v;
            }
            if (++head == p.G) {
              head = 0;
              ++node;
            }
          }
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(p.status, TV_DEV_TIMEOUT);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
}

// ---------------------------------------------------------------- host

template <int D, int N, bool WIN>
cudaError_t launch_t(const AttnParams& p, cudaStream_t st) {
  using C = Cfg<D, N>;
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return cudaErrorInvalidValue;
  CUtensorMap mq;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.R};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * p.Hq};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(N / p.G)}, es[3] = {1, 1, 1};
  if (fn(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const cudaError_t e = ensure_max_dynamic_smem<tv_attn_kv4_kernel<D, N, WIN>>((int)C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dep(tv_attn_kv4_kernel<D, N, WIN>, dim3(p.row_tiles, p.Hkv * p.splits, p.B), dim3(C::kThreads), C::SMEM,
                    st, p, mq);
}

template <int D, bool WIN>
cudaError_t launch_n(const AttnParams& p, int N, cudaStream_t s) {
  if (N == 16) return launch_t<D, 16, WIN>(p, s);
  if (N == 32) return launch_t<D, 32, WIN>(p, s);
  if constexpr (D < 512) {
    if (N == 128) return launch_t<D, 128, WIN>(p, s);
  }
  return launch_t<D, 64, WIN>(p, s);
}

template <bool WIN>
cudaError_t launch_d(const AttnParams& p, int N, cudaStream_t s) {
  if (p.d == 128) return launch_n<128, WIN>(p, N, s);
  if (p.d == 256) return launch_n<256, WIN>(p, N, s);
  return launch_n<512, WIN>(p, N, s);
}

template <int D>
int ctas_of(int N) {
  return N == 16 ? Cfg<D, 16>::CTAS : (N == 32 ? Cfg<D, 32>::CTAS : (N == 64 ? Cfg<D, 64>::CTAS : 1));
}

}  // namespace

bool kv4_tc_supported(const tv_desc* d, int G) { return d->dtype == TV_BF16 && G <= 64; }

// Columns (query rows) of a tile: the smallest of 16, 32, 64 and, up to
// head_dim 256, 128 that holds a sequence's rows.
int kv4_tc_columns(int max_nodes, int G, int d) {
  const int rows = max_nodes * G;
  if (rows <= 16) return 16;
  if (rows <= 32) return 32;
  return rows <= 64 || d == 512 ? 64 : 128;
}

int kv4_tc_ctas_per_sm(int d, int N) { return d == 128 ? ctas_of<128>(N) : (d == 256 ? ctas_of<256>(N) : ctas_of<512>(N)); }

int kv4_tc_key_tile() { return BK; }

cudaError_t launch_attn_kv4(const AttnParams& p, int columns, cudaStream_t s) {
  return p.window > 0 ? launch_d<true>(p, columns, s) : launch_d<false>(p, columns, s);
}

}  // namespace tv
