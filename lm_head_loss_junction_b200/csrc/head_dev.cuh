// Device helpers shared by the single-exit operators' kernels.
#pragma once
#include "common.cuh"

namespace mls {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x, to about 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// l log2(e) - m, rounded once (log2e: head_log2e of the product that made l).
__device__ __forceinline__ float to_base2(float l, float log2e, float m) { return fmaf(l, log2e, -m); }

// The kernels of one call are launched so that the next may be set up while one
// runs; each thread waits here, before its first access to global memory, until
// everything before on the stream is complete and visible.  Loads after it are
// plain ones: a read-only load (__ldg, or of a const __restrict__ pointer) may
// be moved before the wait, where the kernel before still writes.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace mls
