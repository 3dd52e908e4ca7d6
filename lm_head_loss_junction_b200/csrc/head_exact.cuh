// Logits as products summed in 64 bits, and the gradient's entries that need
// them.
//
// The gradient of an entry that holds most of its row is a small difference:
// q (A + B log q) less its coefficient, of the size of 1 - q where a token is
// nearly certain.  Its q comes from a logit and from the forward pass's
// log-sum-exp.  A logit of the tensor cores is off by a few 1e-6 of itself (the
// running sum is truncated at each step), by amounts that differ between the
// kernels for few tokens, for many, and for alternatives, so the difference of
// the two was off by 1e-4 for logits near 45: for q = 0.9999 as much as the
// gradient itself.  With the entry's logit exact in both passes, what is left
// is the rounding of the log-sum-exp to fp32.  (T = 100, D = 2304, W with a mean
// row: dh of rows with q = 0.999 was off by 1.7%, of 0.9999 by 19%; fp32 products
// throughout 0.1% and 1.2%.)
#pragma once
#include <cuda_bf16.h>

#include "head.h"
#include "head_dev.cuh"

namespace mls {

// Products h . W[id[g]] in 64 bits of G rows of W at once (their loads in
// flight together), by one warp, each lane with the results.  w2 (fp32 inputs,
// may be NULL): the rows' squared norms.
template <bool BF16, int G>
__device__ __forceinline__ void dots64(const void* h, const void* W, int64_t D, const int* id, int lane,
                                       double (&acc)[G], float* w2 = nullptr) {
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = 0.0;
  if constexpr (BF16) {
    // a product of two bf16 values is exact in fp32
    const uint4* a = static_cast<const uint4*>(h);
    const uint4* b[G];
#pragma unroll
    for (int g = 0; g < G; ++g) b[g] = static_cast<const uint4*>(W) + id[g] * (D / 8);
    const int n = static_cast<int>(D / 8);
#pragma unroll(G == 1 ? 4 : 1)
    for (int i = lane; i < n; i += 32) {
      uint4 w[G];
#pragma unroll
      for (int g = 0; g < G; ++g) w[g] = b[g][i];
      float x[8];
      bf16x8_to_f32(a[i], x);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float y[8];
        bf16x8_to_f32(w[g], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[g] += static_cast<double>(x[k] * y[k]);
      }
    }
  } else {
    const float* a = static_cast<const float*>(h);
    float sq[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sq[g] = 0.f;
    for (int64_t i = lane; i < D; i += 32) {
      const double x = a[i];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float w = static_cast<const float*>(W)[id[g] * D + i];
        acc[g] = fma(x, static_cast<double>(w), acc[g]);
        sq[g] = fmaf(w, w, sq[g]);
      }
    }
    if (w2 != nullptr) {
#pragma unroll
      for (int g = 0; g < G; ++g) w2[g] = warp_sum(sq[g]);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[g] += __shfl_xor_sync(0xffffffffu, acc[g], o);
}

// The entries [begin, end) of a token (sorted by id, coefficients over the row's
// scale) by one warp.  dense(id, sum of its coefficients): the dense part of G'
// there as it was formed; put(id, G', heavy) once per id, heavy: its dense part
// was formed again from a product in 64 bits (bf16: only then is G' right, the
// others' are in place).  Reading G' of every entry, of 64 teacher tokens each,
// took 45 us at T = 8192; few of them weigh enough.
template <bool BF16, typename Dense, typename Put>
__device__ __forceinline__ void exact_entries(const int2* e, int begin, int end, const float4& ri, const void* h,
                                              const void* W, int64_t D, int lane, const Dense& dense, const Put& put) {
  const bool entropy = ri.z != 0.f;
  const float heavy = fabsf(ri.y) * (1.f / 32);
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    int own = 0;
    float sum = 0.f, was = 0.f;
    bool once = false, some = false;
    if (i < end) {
      own = e[i].x;
      once = i == begin || e[i - 1].x != own;
      if (once) {
        for (int j = i; j < end && e[j].x == own; ++j) sum += __int_as_float(e[j].y);
        // a coefficient that is small beside the row leaves no small difference there; with an entropy's gradient,
        // q (A + B log q) is one itself
        some = entropy || fabsf(sum) > 0.5f * heavy;
        if (some || !BF16) was = dense(own, sum);
      }
    }
    const bool again = entropy ? some : some && fabsf(was) > heavy;
    if (once && !again) put(own, was + sum, false);
    unsigned todo = __ballot_sync(0xffffffffu, again);
    while (todo != 0) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int id[1] = {__shfl_sync(0xffffffffu, own, src)};
      double l[1];
      dots64<BF16, 1>(h, W, D, id, lane, l);
      if (lane == src) {
        // (2^-200 is 0 to ex2; a masked token's d may be infinite)
        const float d = max_nan(static_cast<float>((l[0] - static_cast<double>(ri.x)) * 1.4426950408889634), -200.f);
        put(own, fmaf(ex2(d), fmaf(ri.z * kLn2, d, ri.y), sum), true);
      }
    }
  }
}

}  // namespace mls
