// The 4-bit cache's format (include/tree_kv4.h) in device code: addresses
// inside blocks, scale bytes, and the expansion of a word of eight values.
#pragma once

#include "tv_internal.cuh"

namespace tv {
namespace kv4 {

constexpr int kGroup = 32;                            // channels per K scale

__host__ __device__ constexpr int k_block_bytes(int d) { return 8 * d + d / 2; }
__host__ __device__ constexpr int v_block_bytes(int d) { return 8 * d + 16; }

// offset of position i's 16 bytes of channel group c, and of its scale byte
__device__ __forceinline__ int k_code(int c, int i) { return c * 256 + i * 16; }
__device__ __forceinline__ int k_scale(int d, int c, int i) { return 8 * d + c * 16 + i; }
// offset of channel ch's 8 bytes, and of position i's scale byte
__device__ __forceinline__ int v_code(int ch) { return ch * 8; }
__device__ __forceinline__ int v_scale(int d, int i) { return 8 * d + i; }

// scale byte e * 8 + m as a float: 2^(e - 15) (1 + m / 8), from its bits
__device__ __forceinline__ float scale_of(uint32_t code) { return __uint_as_float((code << 20) + (112u << 23)); }

// the eight values u - 8 of a word (value 2 j at bits 4 j, 2 j + 1 at bits 16 +
// 4 j): a masked pair is two bf16 numbers 128 + u (no conversion instruction)
__device__ __forceinline__ void expand8(uint32_t w, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t pair = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
    x[2 * j] = __uint_as_float(pair << 16) - 136.f;
    x[2 * j + 1] = __uint_as_float(pair & 0xffff0000u) - 136.f;
  }
}

// Expansion in bf16 pairs: a masked pair is 128 + u, and
// (128 + u) s - 136 s = (u - 8) s is one fused multiply-add, exact because s has
// 4 significant bits.  (That a 4-bit code under the exponent of 128 is a number
// is the known way to widen 4-bit weights without a conversion.)
constexpr uint32_t kMinus136 = 0xC308C308u, kOne = 0x3F803F80u, kMinusZero = 0x80008000u;   // bf16 pairs

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Pair j of a word as two bf16 numbers 128 + u: (w >> 4 j) & mask | base, one
// three-input operation with the two constants in registers (as immediates
// they would take two).
struct PairBits {
  uint32_t mask, base;
  __device__ __forceinline__ PairBits() {
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(base));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t w, int j) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * j)), "r"(mask), "r"(base));
    return r;
  }
};

// block `blk` of sequence b and KV head g (paged: through the page table;
// nullptr for a page id out of range)
__device__ __forceinline__ const uint8_t* block_at(const uint8_t* base, int bytes, int b, int g, int64_t blk, int Hkv,
                                                   int64_t max_pages, const int32_t* page_table, int64_t num_pages) {
  if (page_table) {
    const int pid = page_table[(int64_t)b * max_pages + blk];
    if (pid < 0 || pid >= num_pages) return nullptr;
    return base + ((int64_t)pid * Hkv + g) * bytes;
  }
  return base + (((int64_t)b * Hkv + g) * max_pages + blk) * bytes;
}

}  // namespace kv4
}  // namespace tv
