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

// value e of a word: bits 4 j for e = 2 j, 16 + 4 j for e = 2 j + 1
__device__ __forceinline__ int nibble(uint32_t w, int e) { return (int)((w >> ((e >> 1) * 4 + (e & 1) * 16)) & 15u); }

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
