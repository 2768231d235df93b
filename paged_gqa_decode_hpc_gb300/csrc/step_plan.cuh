// What the kernels that plan a step themselves (step_kernel.cu, kv4_decode_kernel.cu)
// have in common: the arithmetic of parts and pool chunks, and the atomic that counts
// a split pair's pieces.
#pragma once
#include <stdint.h>

namespace hpc {
namespace {

// Owner arithmetic of the step plan: parts [0, P) over the first S units,
// then chunks of C units up to T. Every unit index is below T <= INT32_MAX,
// so the arithmetic is 32-bit (short, fast code on a path that runs cold once
// per step); the part formulas take 64 bits only when S * P does not fit.
struct StepMath {
  uint32_t T, S, P, C, chunks;
  bool small;  // (S + 1) * (P + 1) < 2^32
  __device__ __forceinline__ uint32_t part_start(uint32_t o) const {
    return small ? o * S / P : (uint32_t)((uint64_t)o * S / P);
  }
  __device__ __forceinline__ uint32_t start(uint32_t o) const {
    return o < P ? part_start(o) : S + (o - P) * C;
  }
  __device__ __forceinline__ uint32_t end(uint32_t o) const {
    if (o < P) return o + 1 < P ? part_start(o + 1) : S;
    const uint32_t e = S + (o - P + 1) * C;
    return e < T ? e : T;
  }
  __device__ __forceinline__ uint32_t owner_of(uint32_t x) const {
    if (x < S) return small ? ((x + 1) * P - 1) / S : (uint32_t)(((uint64_t)(x + 1) * P - 1) / S);
    return P + (x - S) / C;
  }
};

// atomicAdd with acquire-release semantics at device scope: the writes that
// happen before it (this thread's, and the warp's through a warp barrier)
// are visible before the addition, and reads after it see what the earlier
// releasers wrote.
__device__ __forceinline__ int atom_add_acq_rel_gpu(int32_t* p, int v) {
  int prev;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(prev) : "l"(p), "r"(v)
               : "memory");
  return prev;
}

}  // namespace
}  // namespace hpc
