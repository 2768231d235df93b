// Small inline-PTX helpers shared by the library's kernels.
#pragma once
#include <stdint.h>

namespace hpc {

__device__ __forceinline__ float ptx_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Programmatic dependent launch: wait until the preceding kernel in the
// stream has completed and its memory is visible (a no-op when this kernel
// was launched without the programmatic-serialization attribute).
__device__ __forceinline__ void griddep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Let the next kernel in the stream start launching its CTAs.
__device__ __forceinline__ void griddep_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Registers a thread of this warpgroup from here on: more, out of what the CTA was launched
// with and others have given back, or fewer.
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N) : "memory");
}

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

}  // namespace hpc
