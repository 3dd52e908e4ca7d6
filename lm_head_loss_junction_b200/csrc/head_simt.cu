// fp32 path of the single-exit LM-head operators: CUDA-core matrix products
// (tensor cores would round fp32 inputs), logits of a block of tokens in the
// workspace, any sizes.  For the small single-precision suite; bound by
// latency there (a handful of 64 x 64 tiles).
#include "head.h"
#include "head_dev.cuh"

namespace mls {

namespace {

constexpr int kTile = 64, kK = 16, kThreads = 256;

// C[m][n] = sum_k A(m, k) B(n, k) (+ C).  A_K / B_K: k is the operand's
// contiguous dimension (row stride lda), otherwise m / n is.  64 x 64 tiles,
// 4 x 4 outputs per thread, the next K slice loaded into registers while the
// current one is multiplied.  krow (with !B_K): rows k of B whose .w is 0 count
// as zeros, whatever they hold.
template <bool A_K, bool B_K>
__global__ void __launch_bounds__(kThreads) sgemm_kernel(const float* __restrict__ A, int64_t lda,
                                                         const float* __restrict__ B, int64_t ldb,
                                                         float* __restrict__ C, int64_t ldc, int M, int N, int K,
                                                         int accumulate, const float4* __restrict__ krow) {
  __shared__ float sa[2][kK][kTile + 4], sb[2][kK][kTile + 4];
  const int tid = threadIdx.x;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  float ra[4], rb[4];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = i * kThreads + tid;
      const int ak = A_K ? e % kK : e / kTile, am = A_K ? e / kK : e % kTile;
      const int bk = B_K ? e % kK : e / kTile, bn = B_K ? e / kK : e % kTile;
      const int64_t am_g = m0 + am, bn_g = n0 + bn;
      ra[i] = am_g < M && k0 + ak < K ? __ldg(A + (A_K ? am_g * lda + k0 + ak : (k0 + ak) * lda + am_g)) : 0.f;
      const bool live = bn_g < N && k0 + bk < K && (B_K || krow == nullptr || krow[k0 + bk].w != 0.f);
      rb[i] = live ? __ldg(B + (B_K ? bn_g * ldb + k0 + bk : (k0 + bk) * ldb + bn_g)) : 0.f;
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = i * kThreads + tid;
      sa[buf][A_K ? e % kK : e / kTile][A_K ? e / kK : e % kTile] = ra[i];
      sb[buf][B_K ? e % kK : e / kTile][B_K ? e / kK : e % kTile] = rb[i];
    }
  };
  const int tx = tid % 16, ty = tid / 16;
  float acc[4][4] = {};
  fetch(0);
  put(0);
  __syncthreads();
  int buf = 0;
  for (int k0 = 0; k0 < K; k0 += kK) {
    const bool more = k0 + kK < K;
    if (more) fetch(k0 + kK);
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&sa[buf][k][ty * 4]);
      const float4 b = *reinterpret_cast<const float4*>(&sb[buf][k][tx * 4]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    if (more) put(buf ^ 1);
    __syncthreads();
    buf ^= 1;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (n >= N) continue;
      float* c = C + m * ldc + n;
      *c = accumulate ? *c + acc[i][j] : acc[i][j];
    }
  }
}

template <bool A_K, bool B_K>
cudaError_t sgemm(const float* A, int64_t lda, const float* B, int64_t ldb, float* C, int64_t ldc, int64_t M,
                  int64_t N, int64_t K, int accumulate, const float4* krow, cudaStream_t st) {
  // grid.y is at most 65535: longer outputs go in pieces of rows
  const int64_t most = int64_t(65535) * kTile;
  for (int64_t r = 0; r < M; r += most) {
    const int64_t rows = M - r < most ? M - r : most;
    const dim3 grid(static_cast<unsigned>((N + kTile - 1) / kTile), static_cast<unsigned>((rows + kTile - 1) / kTile));
    sgemm_kernel<A_K, B_K><<<grid, kThreads, 0, st>>>(A_K ? A + r * lda : A + r, lda, B, ldb, C + r * ldc, ldc,
                                                      static_cast<int>(rows), static_cast<int>(N),
                                                      static_cast<int>(K), accumulate, krow);
    note_launches(1);
  }
  return cudaGetLastError();
}

// One warp per (token, split).
__global__ void __launch_bounds__(256) split_stats_kernel(const float* __restrict__ logits, int64_t ld, int64_t T,
                                                          int V, int n_splits, HeadPart* __restrict__ part) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (i >= T * n_splits) return;
  const int64_t t = i / n_splits;
  const int c0 = static_cast<int>(i % n_splits) * kHeadSplit;
  float l[4], top = -INFINITY, z = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int col = c0 + k * 32 + lane;
    l[k] = col < V ? logits[t * ld + col] : -INFINITY;
    top = fmaxf(top, l[k]);
  }
  top = warp_max(top);
  const float m = top * kLog2e;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c0 + k * 32 + lane >= V) continue;
    const float d = to_base2(l[k], m), e = ex2(d);
    z += e;
    u = fmaf(d, e, u);
  }
  z = warp_sum(z);
  u = warp_sum(u);
  if (lane == 0) part[i] = make_float4(m, z, u, top);
}

// Logits -> s (q (A + B (l - lse)) + entries) in place, one block per token.
__global__ void __launch_bounds__(256) grad_rows_kernel(float* __restrict__ logits, int64_t ld, int V,
                                                        const HeadEntries en, int64_t t0, int64_t T, int n_splits) {
  const int64_t t = t0 + blockIdx.x;
  float* row = logits + static_cast<int64_t>(blockIdx.x) * ld;
  const float4 ri = en.row[t];
  for (int v = threadIdx.x; v < V; v += 256) {
    const float d = to_base2(row[v], ri.x * kLog2e);
    row[v] = ri.w == 0.f ? 0.f : ri.w * (ex2(d) * fmaf(ri.z * kLn2, d, ri.y));
  }
  __syncthreads();
  if (threadIdx.x == 0 && ri.w != 0.f) {
    const int n = en.first[static_cast<int64_t>(n_splits) * T + t];
    for (int i = 0; i < n; ++i) {
      const int2 e = en.e[t * en.Ntot + i];
      row[e.x] += ri.w * __int_as_float(e.y);
    }
  }
}

}  // namespace

cudaError_t head_simt_logits(const HeadProblem& p, int64_t t0, int64_t Tb, float* logits, int64_t ld, HeadPart* part,
                             cudaStream_t st) {
  const float* h = static_cast<const float*>(p.h) + t0 * p.D;
  cudaError_t err = sgemm<true, true>(h, p.D, static_cast<const float*>(p.W), p.D, logits, ld, Tb, p.V, p.D, 0,
                                      nullptr, st);
  if (err != cudaSuccess || part == nullptr) return err;
  const int64_t n = head_splits(p.V);
  split_stats_kernel<<<static_cast<unsigned>((Tb * n + 7) / 8), 256, 0, st>>>(logits, ld, Tb, static_cast<int>(p.V),
                                                                              static_cast<int>(n), part);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t head_simt_backward(const HeadProblem& p, const HeadEntries& en, float* dh, float* dW, int accumulate,
                               float* logits, int64_t Tb, cudaStream_t st) {
  const float* W = static_cast<const float*>(p.W);
  const int64_t ld = p.V;
  for (int64_t t0 = 0; t0 < p.T; t0 += Tb) {
    const int64_t n = t0 + Tb <= p.T ? Tb : p.T - t0;
    cudaError_t err = head_simt_logits(p, t0, n, logits, ld, nullptr, st);
    if (err != cudaSuccess) return err;
    grad_rows_kernel<<<static_cast<unsigned>(n), 256, 0, st>>>(logits, ld, static_cast<int>(p.V), en, t0, p.T,
                                                               static_cast<int>(head_splits(p.V)));
    note_launches(1);
    if (dh != nullptr) {
      err = sgemm<true, false>(logits, ld, W, p.D, dh + t0 * p.D, p.D, n, p.D, p.V, 0, nullptr, st);
      if (err != cudaSuccess) return err;
    }
    if (dW != nullptr) {
      err = sgemm<false, false>(logits, ld, static_cast<const float*>(p.h) + t0 * p.D, p.D, dW, p.D, p.V, p.D, n,
                                accumulate != 0 || t0 > 0, en.row + t0, st);
      if (err != cudaSuccess) return err;
    }
  }
  return cudaGetLastError();
}

}  // namespace mls
