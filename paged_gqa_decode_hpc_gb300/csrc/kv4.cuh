// Device pieces of the 4-bit cache shared by the kernels that read and write it.
//
// A row (one token's K or V of one KV head) is 72 bytes: 64 of e2m1 codes, element
// 2i of the head in the low four bits of byte i and 2i + 1 in the high ones, then
// eight e4m3 scales, scale j of elements 16 j .. 16 j + 15. A (block, KV head) tile
// is its 64 rows, 4608 contiguous bytes. An element stands for code * scale * (the
// tensor's own scale); the product of an e2m1 and an e4m3 has six significant bits
// and is a multiple of 2^-10 of at most 2688, so it is an f16 value: kernels multiply
// the two in f16 exactly and keep the tensor's scale for the end.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace hpc {

constexpr int kKv4Row = 72;                  // bytes of a row
constexpr int kKv4Codes = 64;                // of codes, ahead of the scales
constexpr int kKv4Span = 16;                 // elements that share a scale
constexpr int kKv4Tile = 64 * kKv4Row;       // one (block, KV head) tile of K or of V

#ifdef __CUDACC__

// What the copies of a tile read where the block table holds no valid block.
static __device__ const uint4 kKv4NoTile[kKv4Tile / 16] = {};

// Eight e2m1 codes to f16, exactly: byte i of x becomes the pair r[i] (low code in
// the low half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t x, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(x));
}

// Two e4m3 scales (low byte -> low half) to f16, exactly.
__device__ __forceinline__ uint32_t kv4_scales(uint32_t x) {
  uint32_t r;
  const uint16_t h = (uint16_t)x;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A pair's low or high half in both halves.
__device__ __forceinline__ uint32_t both_low(uint32_t a) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, 0x1010;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t both_high(uint32_t a) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, 0x3232;" : "=r"(r) : "r"(a));
  return r;
}

// One tile to shared memory: 16-byte aligned at both ends.
__device__ __forceinline__ void kv4_copy_tile(uint32_t dst, const void* src, uint32_t bar,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(__cvta_generic_to_global(src)), "r"((uint32_t)kKv4Tile), "r"(bar), "l"(policy)
      : "memory");
}

// Any multiple of 16 bytes.
__device__ __forceinline__ void kv4_copy(uint32_t dst, const void* src, uint32_t bytes,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

#endif  // __CUDACC__

}  // namespace hpc
