// fp32 path of the single-exit LM-head operators: CUDA-core matrix products
// (tensor cores would round fp32 inputs), logits of a block of tokens in the
// workspace, any sizes.  For the small single-precision suite; bound by
// latency there (one tile of 16 x 16 or 32 x 32 per SM).
#include "head.h"
#include "head_dev.cuh"
#include "head_exact.cuh"
#include "head_host.h"

namespace mls {

namespace {

constexpr int kThreads = 256;

// C[m][n] = sum_k A(m, k) B(n, k) (+ C).  A_K / B_K: k is the operand's
// contiguous dimension (row stride lda), otherwise m / n is.  TILE x TILE
// outputs per block, 4 x 4 per thread; with TILE = 32 (16) the block's 4 (16)
// groups of threads take a part of K each and their sums are added in order.
// The next K slice is loaded into registers while the current one is
// multiplied.  krow (with !B_K): rows k of B whose .w is 0 count as zeros,
// whatever they hold.
template <bool A_K, bool B_K, int TILE>
__global__ void __launch_bounds__(kThreads) sgemm_kernel(const float* A, int64_t lda,
                                                         const float* B, int64_t ldb,
                                                         float* C, int64_t ldc, int M, int N, int K,
                                                         int accumulate, const float4* krow) {
  constexpr int kK = TILE == 16 ? 16 : 32;               // K per slice
  constexpr int kPer = (TILE / 4) * (TILE / 4);          // threads of a group
  constexpr int kGroups = kThreads / kPer;
  constexpr int kLd = TILE * kK / kPer;                  // values of each operand per thread and slice
  __shared__ __align__(16) float sa[kGroups][kK][TILE + 4], sb[kGroups][kK][TILE + 4];
  after_previous();
  const int group = threadIdx.x / kPer, tid = threadIdx.x % kPer;
  const int m0 = blockIdx.y * TILE, n0 = blockIdx.x * TILE;
  const int per = (K + kGroups * kK - 1) / (kGroups * kK) * kK;
  const int k_begin = group * per, k_end = min(K, k_begin + per);
  float ra[kLd], rb[kLd];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kLd; ++i) {
      const int e = i * kPer + tid;
      const int ak = A_K ? e % kK : e / TILE, am = A_K ? e / kK : e % TILE;
      const int bk = B_K ? e % kK : e / TILE, bn = B_K ? e / kK : e % TILE;
      const int64_t am_g = m0 + am, bn_g = n0 + bn;
      ra[i] = am_g < M && k0 + ak < k_end ? A[A_K ? am_g * lda + k0 + ak : (k0 + ak) * lda + am_g] : 0.f;
      const bool live = bn_g < N && k0 + bk < k_end && (B_K || krow == nullptr || krow[k0 + bk].w != 0.f);
      rb[i] = live ? B[B_K ? bn_g * ldb + k0 + bk : (k0 + bk) * ldb + bn_g] : 0.f;
    }
  };
  auto put = [&]() {
#pragma unroll
    for (int i = 0; i < kLd; ++i) {
      const int e = i * kPer + tid;
      sa[group][A_K ? e % kK : e / TILE][A_K ? e / kK : e % TILE] = ra[i];
      sb[group][B_K ? e % kK : e / TILE][B_K ? e / kK : e % TILE] = rb[i];
    }
  };
  const int tx = tid % (TILE / 4), ty = tid / (TILE / 4);
  float acc[4][4] = {};
  fetch(k_begin);
  for (int k = 0; k < per; k += kK) {
    put();
    __syncthreads();
    if (k + kK < per) fetch(k_begin + k + kK);
#pragma unroll
    for (int j = 0; j < kK; ++j) {
      const float4 a = *reinterpret_cast<const float4*>(&sa[group][j][ty * 4]);
      const float4 b = *reinterpret_cast<const float4*>(&sb[group][j][tx * 4]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int l = 0; l < 4; ++l) acc[i][l] = fmaf(av[i], bv[l], acc[i][l]);
    }
    __syncthreads();
  }
  if constexpr (kGroups > 1) {
    // the groups' sums meet in shared memory (the slices are read no more)
    float* sums = &sa[0][0][0];
    static_assert(sizeof(sa) >= (kGroups - 1) * TILE * TILE * sizeof(float), "room for the sums");
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[(group - 1) * TILE * TILE + i * kPer + tid] = acc[i / 4][i % 4];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < kGroups - 1; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i / 4][i % 4] += sums[g * TILE * TILE + i * kPer + tid];
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

template <bool A_K, bool B_K, int TILE>
cudaError_t sgemm_tiles(const float* A, int64_t lda, const float* B, int64_t ldb, float* C, int64_t ldc, int64_t M,
                        int64_t N, int64_t K, int accumulate, const float4* krow, cudaStream_t st) {
  // grid.y is at most 65535: longer outputs go in pieces of rows
  const int64_t most = int64_t(65535) * TILE;
  for (int64_t r = 0; r < M; r += most) {
    const int64_t rows = M - r < most ? M - r : most;
    const dim3 grid(static_cast<unsigned>((N + TILE - 1) / TILE), static_cast<unsigned>((rows + TILE - 1) / TILE));
    const cudaError_t err =
        head_launch(sgemm_kernel<A_K, B_K, TILE>, grid, kThreads, 0, st, A_K ? A + r * lda : A + r, lda, B, ldb,
                    C + r * ldc, ldc, static_cast<int>(rows), static_cast<int>(N), static_cast<int>(K), accumulate, krow);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// The largest tiles that give every SM one, or every other SM one of 32 x 32
// (M = 256, N = 128, K = 512: 8 blocks of 64 x 64 took 33 us, 32 of 32 x 32
// 15 us, 128 of 16 x 16 7.5 us; M = 256, N = 512, K = 192: 128 of 32 x 32 5 us,
// 512 of 16 x 16 8.5 us).  all: the rows of the whole
// problem, of which M may be a piece: the sums of a row do not depend on the
// pieces.
template <bool A_K, bool B_K>
cudaError_t sgemm(const float* A, int64_t lda, const float* B, int64_t ldb, float* C, int64_t ldc, int64_t M,
                  int64_t N, int64_t K, int accumulate, const float4* krow, int64_t all, cudaStream_t st) {
  if (((all + 63) / 64) * ((N + 63) / 64) >= 148)
    return sgemm_tiles<A_K, B_K, 64>(A, lda, B, ldb, C, ldc, M, N, K, accumulate, krow, st);
  if (((all + 31) / 32) * ((N + 31) / 32) >= 74)
    return sgemm_tiles<A_K, B_K, 32>(A, lda, B, ldb, C, ldc, M, N, K, accumulate, krow, st);
  return sgemm_tiles<A_K, B_K, 16>(A, lda, B, ldb, C, ldc, M, N, K, accumulate, krow, st);
}

// One warp per (token, split).
__global__ void __launch_bounds__(256) split_stats_kernel(const float* logits, int64_t ld, int64_t T,
                                                          int V, int n_splits, HeadPart* part) {
  after_previous();
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
  const bool large = fabsf(top) > kLarge;
  const float low = fmaxf(top, kLowest), m = (large ? low : top) * kLog2e;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c0 + k * 32 + lane >= V) continue;
    const float d = large ? low_base2(l[k], kLog2e, low) : max_nan(to_base2(l[k], kLog2e, m), -200.f), e = ex2(d);
    z += e;
    u = fmaf(d, e, u);
  }
  z = warp_sum(z);
  u = warp_sum(u);
  if (lane == 0) part[i] = make_float4(m, z, u, top);
}

// Logits -> s (q (A + B (l - lse)) + entries) in place, one block per token; h: the
// rows of the block of tokens.
__global__ void __launch_bounds__(256) grad_rows_kernel(float* logits, int64_t ld, int V, const HeadEntries en,
                                                        const float* h, const float* W, int64_t D, int64_t t0, int64_t T,
                                                        int n_splits) {
  after_previous();
  const int64_t t = t0 + blockIdx.x;
  float* row = logits + static_cast<int64_t>(blockIdx.x) * ld;
  const float4 ri = en.row[t];
  for (int v = threadIdx.x; v < V; v += 256) {
    // the difference first: rounding lse log2(e) would cost every q of the row 1e-6 of itself
    const float d = max_nan((row[v] - ri.x) * kLog2e, -200.f);
    row[v] = ri.w == 0.f ? 0.f : ri.w * (ex2(d) * fmaf(ri.z * kLn2, d, ri.y));
  }
  __syncthreads();
  if (threadIdx.x < 32 && ri.w != 0.f) {
    const float over = 1.f / ri.w;
    exact_entries<false>(
        en.e + t * en.Ntot, 0, en.first[static_cast<int64_t>(n_splits) * T + t], ri,
        h + static_cast<int64_t>(blockIdx.x) * D, W, D, threadIdx.x, [&](int id, float) { return row[id] * over; },
        [&](int id, float v, bool) { row[id] = ri.w * v; });
  }
}

}  // namespace

cudaError_t head_simt_logits(const HeadProblem& p, int64_t t0, int64_t Tb, float* logits, int64_t ld, HeadPart* part,
                             cudaStream_t st) {
  const float* h = static_cast<const float*>(p.h) + t0 * p.D;
  cudaError_t err = sgemm<true, true>(h, p.D, static_cast<const float*>(p.W), p.D, logits, ld, Tb, p.V, p.D, 0,
                                      nullptr, p.T, st);
  if (err != cudaSuccess || part == nullptr) return err;
  const int64_t n = head_splits(p.V);
  return head_launch(split_stats_kernel, dim3(static_cast<unsigned>((Tb * n + 7) / 8)), 256, 0, st, logits, ld, Tb,
                     static_cast<int>(p.V), static_cast<int>(n), part);
}

cudaError_t head_simt_backward(const HeadProblem& p, const HeadEntries& en, float* dh, float* dW, int accumulate,
                               float* logits, int64_t Tb, cudaStream_t st) {
  const float* W = static_cast<const float*>(p.W);
  const int64_t ld = p.V;
  for (int64_t t0 = 0; t0 < p.T; t0 += Tb) {
    const int64_t n = t0 + Tb <= p.T ? Tb : p.T - t0;
    cudaError_t err = head_simt_logits(p, t0, n, logits, ld, nullptr, st);
    if (err != cudaSuccess) return err;
    err = head_launch(grad_rows_kernel, dim3(static_cast<unsigned>(n)), 256, 0, st, logits, ld, static_cast<int>(p.V),
                      en, static_cast<const float*>(p.h) + t0 * p.D, W, p.D, t0, p.T, static_cast<int>(head_splits(p.V)));
    if (err != cudaSuccess) return err;
    if (dh != nullptr) {
      err = sgemm<true, false>(logits, ld, W, p.D, dh + t0 * p.D, p.D, n, p.D, p.V, 0, nullptr, p.T, st);
      if (err != cudaSuccess) return err;
    }
    if (dW != nullptr) {
      err = sgemm<false, false>(logits, ld, static_cast<const float*>(p.h) + t0 * p.D, p.D, dW, p.D, p.V, p.D, n,
                                accumulate != 0 || t0 > 0, en.row + t0, p.V, st);
      if (err != cudaSuccess) return err;
    }
  }
  return cudaSuccess;
}

}  // namespace mls
