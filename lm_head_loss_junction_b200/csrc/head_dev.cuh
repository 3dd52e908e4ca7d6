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

// The larger of the two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (m, z, u) of two column sets -> of their union: with d = m - m', a' = a + d,
// 2^a' = 2^d 2^a.  A set that vanishes beside the other has no u left (its d may
// be infinite).
__device__ __forceinline__ void merge_part(float& m, float& z, float& u, float m2, float z2, float u2) {
  const float top = fmaxf(m, m2);
  if (!(top > -INFINITY)) {                              // nothing on either side, or nothing that is a number
    z += z2;
    u += u2;
    return;
  }
  if (z > 0.f || z != z) {
    const float d = m - top, f = ex2(d);
    u = f > 0.f ? f * fmaf(d, z, u) : 0.f;
    z *= f;
  }
  if (z2 > 0.f || z2 != z2) {
    const float d = m2 - top, f = ex2(d);
    if (f > 0.f) u = fmaf(f, fmaf(d, z2, u2), u);
    z = fmaf(f, z2, z);
  }
  m = top;
}

// Pieces of a row whose largest logit is as far from 0 as a mask (or passes
// kLarge for another reason): l log2(e) - m would be off by the rounding of m, or
// overflow.  They are summed over their largest logit itself, which its rounded m
// then stands for; nothing lies below kLowest.  A single logit that low in another
// piece is only kept from the infinite (2^-200 is 0 to ex2).
constexpr float kLarge = 1.0e6f;
constexpr float kLowest = -2.3e38f;          // times log2(e) it is finite
__device__ __forceinline__ float low_base2(float l, float log2e, float top) {
  return max_nan((max_nan(l, kLowest) - top) * log2e, -200.f);
}

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
