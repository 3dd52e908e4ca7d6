// fp16 copies of W and h.  kind::f16 takes A and B of one type, so G' in fp16
// needs W and h in fp16.  bf16's 8 significant bits fit in fp16's 11: values in
// its normal range convert exactly.
#pragma once
#include "head.h"
#include "head_dev.cuh"

namespace mls {

// h is copied times s_t over the bound on s_t |h|, so that dW can sum the rows
// of G', each over its s_t; times 2^14, so that rows down to 2^-28 of the
// largest stay in fp16's normal range and none passes it.
constexpr float kRowLift = 16384.f;

__device__ __forceinline__ uint4 to_half8(const uint4& v, float f, float& mx) {
  float x[8];
  bf16x8_to_f32(v, x);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // a row of scale 0 is left out, whatever it holds
    const float lo = f == 0.f ? 0.f : x[2 * k] * f, hi = f == 0.f ? 0.f : x[2 * k + 1] * f;
    mx = fmaxf(mx, fmaxf(fabsf(lo), fabsf(hi)));
    __half2 h = __floats2half2_rn(lo, hi);
    w[k] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Thread `first` of `stride` threads (whole warps): the unscaled copy of W, and
// its largest magnitude.
__device__ __forceinline__ void copy_w(const HeadCopyW& a, int64_t first, int64_t stride) {
  const uint4* src = static_cast<const uint4*>(a.src);
  uint4* dst = reinterpret_cast<uint4*>(a.dst);
  float mx = 0.f;
  int64_t i = first;
  for (; i + 7 * stride < a.n_vec; i += 8 * stride) {
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = src[i + k * stride];
#pragma unroll
    for (int k = 0; k < 8; ++k) dst[i + k * stride] = to_half8(v[k], 1.f, mx);
  }
  for (; i < a.n_vec; i += stride) dst[i] = to_half8(src[i], 1.f, mx);
  mx = warp_max(mx);
  if ((threadIdx.x & 31) == 0 && mx > 0.f) atomicMax(a.maxbits, __float_as_uint(mx));
}

// The copy again with a power-of-two scale when the largest magnitude is at or
// past 2^15 or below 2^-6; the reciprocal of the scale for the epilogue.
__device__ __forceinline__ void rescale_w(const HeadCopyW& a, int64_t first, int64_t stride) {
  if (a.n_vec == 0) return;
  const float mx = __uint_as_float(*a.maxbits);
  float s = 1.f;
  if (mx <= 3.4e38f && (mx >= 32768.f || (mx > 0.f && mx < 1.f / 64.f))) {
    int e = 13 - ilogbf(mx);
    e = e < -126 ? -126 : (e > 126 ? 126 : e);
    s = ldexpf(1.f, e);
  }
  if (first == 0) *a.inv = 1.f / s;
  if (s == 1.f) return;
  float unused = 0.f;
  for (int64_t i = first; i < a.n_vec; i += stride)
    reinterpret_cast<uint4*>(a.dst)[i] = to_half8(static_cast<const uint4*>(a.src)[i], s, unused);
}

__device__ __forceinline__ void copy_h(const HeadCopyH& a, int64_t first, int64_t stride) {
  if (a.n_vec == 0) return;
  const uint4* src = static_cast<const uint4*>(a.src);
  uint4* dst = reinterpret_cast<uint4*>(a.dst);
  const float smax = __uint_as_float(*a.smax);
  const auto factor = [&](int64_t i) {
    return smax > 0.f ? a.row[i / a.vec_per_row].w / smax * kRowLift : 0.f;
  };
  float unused = 0.f;
  int64_t i = first;
  for (; i + 3 * stride < a.n_vec; i += 4 * stride) {
    uint4 v[4];
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = src[i + k * stride];
      f[k] = factor(i + k * stride);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[i + k * stride] = to_half8(v[k], f[k], unused);
  }
  for (; i < a.n_vec; i += stride) dst[i] = to_half8(src[i], factor(i), unused);
}

}  // namespace mls
