// Per-token kernels of the single-exit LM-head operators: the entry lists, the
// merge of the partial statistics, and the top alternatives.
#include <cuda_bf16.h>
#include <type_traits>

#include "head.h"
#include "head_copy.cuh"
#include "head_dev.cuh"
#include "head_exact.cuh"
#include "head_host.h"

namespace mls {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------ entry lists
// One warp per token turns the token's ids into a list sorted by id (ties by
// position), with the position (forward) or the coefficient over the row scale
// (backward); then the block's threads write the first entry of every split,
// eight tokens' bytes together.  Bound by the latency of its few dependent
// steps, so a token is a warp's only one (four in turn, with 32 lanes along the
// tokens in the table, took four times as long).
constexpr int kEntryTokens = 8;
constexpr int kMaxTot = kMaxEntries + 1;
constexpr int kPerLane = (kMaxTot + 31) / 32;

constexpr int kPadTot = (kMaxTot + 3) / 4 * 4;

struct EntrySmem {
  uint32_t key[kEntryTokens][kPadTot];
  int sorted[kEntryTokens][kMaxTot];
  int count[kEntryTokens];
};

// The power of two s_t that brings a row of G into [2^14, 2^15) at its bound:
// G' = G / s_t fills fp16's range from the top, so a probability keeps 11 bits
// down to 2^-28 of the bound and counts down to 2^-39.  (With the bound brought
// to 1, what fell below 2^-24 of it was lost: a row's small probabilities all
// have one sign, and of a row with q_y = 0.9997 over 49152 columns half the
// gradient went.)  1 where the bound is no number, which the row then shows.
__device__ __forceinline__ float row_scale(float bound) {
  if (!(bound > 0.f)) return bound == 0.f ? 0.f : 1.f;
  int e = ilogbf(fminf(bound, 3.4e38f)) - 14;
  e = e < -126 ? -126 : e;
  return ldexpf(1.f, e);
}

// Blocks past the tokens' make the fp16 copy of W that dh will read.
__global__ void __launch_bounds__(256) head_entries_kernel(const HeadEntriesIn in, const HeadEntries out,
                                                           bool backward, int n_splits, unsigned token_blocks,
                                                           const HeadCopyW w_copy, int32_t* status) {
  __shared__ __align__(16) EntrySmem s;
  after_previous();
  if (blockIdx.x >= token_blocks) {
    copy_w(w_copy, static_cast<int64_t>(blockIdx.x - token_blocks) * 256 + threadIdx.x,
           static_cast<int64_t>(gridDim.x - token_blocks) * 256);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kEntryTokens;
  const int N = in.N, tot = out.Ntot;
  const int i = warp;
  if (t0 + i < in.T) {
    const int64_t t = t0 + i;
    int id[kPerLane];
    float c[kPerLane];
    bool there[kPerLane];
    bool bad = false;
    float h_most = 0.f;
    if (backward && in.h != nullptr) {
      const uint4* row = static_cast<const uint4*>(in.h) + t * (in.D / 8);
      for (int64_t j = lane; j < in.D / 8; j += 32) {
        float x[8];
        bf16x8_to_f32(row[j], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) h_most = fmaxf(h_most, fabsf(x[k]));
      }
    }
    const float w = in.weights != nullptr ? in.weights[t] : 1.f;
    const int32_t y = in.y != nullptr ? in.y[t] : 0;
    // a token with a bad target is left out; one of weight 0 has no gradient, but terms of its own in stats
    const bool out_y = in.y != nullptr && (y < 0 || y >= in.V);
    const bool skip = out_y || (backward && w == 0.f);
    if (out_y && w != 0.f) bad = true;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int j = k * 32 + lane;
      id[k] = -1;
      c[k] = 0.f;
      if (j < N) {
        id[k] = in.ids[t * N + j];
        if (id[k] != -1 && (id[k] < 0 || id[k] >= in.V)) bad = true;
      } else if (j == N && in.y != nullptr) {
        id[k] = y;
      }
      there[k] = !skip && j < tot && id[k] >= 0 && id[k] < in.V;
    }
    float A = 0.f, B = 0.f, scale = 0.f;
    if (backward) {
      float bound = 0.f;                   // on |G| of the row
      if (in.y == nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          if (there[k]) c[k] = in.g_logp[t * N + k * 32 + lane];
          sum += c[k];
          bound += fabsf(c[k]);
        }
        sum = warp_sum(sum);
        B = in.g_entropy != nullptr ? -in.g_entropy[t] : 0.f;
        A = -sum + (in.g_entropy != nullptr ? B * in.stats[in.T + t] : 0.f);
        // q (H + log q) is largest where one token holds about half and the rest is flat: under 7 for V < 2^31
        bound = warp_sum(bound) + fabsf(sum) + 7.f * fabsf(B);
      } else {
        float z[kPerLane], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          const int j = k * 32 + lane;
          z[k] = there[k] && j < N ? in.teacher[t * N + j] : -INFINITY;
          top = fmaxf(top, z[k]);
        }
        top = warp_max(top);
        const bool some = top > -INFINITY;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          z[k] = some && there[k] && k * 32 + lane < N ? expf(z[k] - top) : 0.f;
          sum += z[k];
        }
        sum = warp_sum(sum);
        const float wg = skip ? 0.f : w * in.grad;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          const int j = k * 32 + lane;
          if (there[k]) c[k] = j == N ? -wg * (1.f - in.alpha) : (some ? -wg * in.alpha * (z[k] / sum) : 0.f);
          bound += fabsf(c[k]);
        }
        A = wg * ((1.f - in.alpha) + (some ? in.alpha : 0.f));
        bound = warp_sum(bound) + fabsf(A);
      }
      scale = row_scale(bound);
      if (lane == 0) {
        const float r = scale != 0.f ? 1.f / scale : 0.f;
        out.row[t] = make_float4(in.stats[t], A * r, B * r, scale);
      }
      if (in.h != nullptr) {
        // a power of two above s |h| (a row of zeros, or of nothing that is a number, counts as 1)
        h_most = warp_max(h_most);
        if (lane == 0 && scale > 0.f) {
          // at least 2^-111 s: s over it, times the lift of the copy (2^14), stays in range for subnormal h too
          const int h_exp = h_most > 0.f && h_most <= 3.4e38f ? max(ilogbf(h_most) + 1, -111) : 0;
          const int e = min(max(ilogbf(scale) + h_exp, -126), 126);
          atomicMax(out.smax, __float_as_uint(ldexpf(1.f, e)));
        }
      }
    }
    if (__any_sync(kFull, bad) && lane == 0) set_flag(status, MLS_DEVFLAG_BAD_ID);
    // rank by (id, position): in one word where the id leaves room for the position, else in two steps
    const bool packed = in.V <= (int64_t(1) << 25);
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int j = k * 32 + lane;
      n += __popc(__ballot_sync(kFull, there[k]));
      const uint32_t word = packed ? static_cast<uint32_t>(id[k]) << 7 | j : static_cast<uint32_t>(id[k]);
      if (j < kPadTot) s.key[i][j] = there[k] ? word : 0xffffffffu;
    }
    if (lane == 0) s.count[i] = n;
    __syncwarp();
    const float r = scale != 0.f ? 1.f / scale : 0.f;
    int rank[kPerLane];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) rank[k] = 0;
    if (packed) {
      for (int o = 0; o < tot; o += 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(&s.key[i][o]);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          const uint32_t mine = static_cast<uint32_t>(id[k]) << 7 | (k * 32 + lane);
          rank[k] += (w.x < mine) + (w.y < mine) + (w.z < mine) + (w.w < mine);
        }
      }
    } else {
      for (int o = 0; o < tot; ++o) {
        const uint32_t w = s.key[i][o];
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          const uint32_t mine = static_cast<uint32_t>(id[k]);
          rank[k] += w < mine || (w == mine && o < k * 32 + lane);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      if (!there[k]) continue;
      s.sorted[i][rank[k]] = id[k];
      out.e[t * tot + rank[k]] = make_int2(id[k], backward ? __float_as_int(c[k] * r) : k * 32 + lane);
    }
  }
  __syncthreads();
  // each thread walks a range of splits of one token: one search, then steps
  const int own = threadIdx.x % kEntryTokens;
  const int64_t t = t0 + own;
  if (t < in.T) {
    const int n = s.count[own];
    const int per = (n_splits + 256 / kEntryTokens) / (256 / kEntryTokens);
    const int begin = threadIdx.x / kEntryTokens * per, end = min(begin + per, n_splits + 1);
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s.sorted[own][mid] < static_cast<int64_t>(begin) * kHeadSplit) lo = mid + 1; else hi = mid;
    }
    for (int sp = begin; sp < end; ++sp) {
      while (lo < n && s.sorted[own][lo] < static_cast<int64_t>(sp) * kHeadSplit) ++lo;
      out.first[static_cast<int64_t>(sp) * in.T + t] = static_cast<uint8_t>(lo);
    }
  }
}

// ------------------------------------------------------------------ entries of the gradient that hold much of a row
// G' of a chunk's entries again where they hold more than about 2^-5 of their
// row, from products in 64 bits (head_exact.cuh).  Blocks past the tokens' give
// the chunk's fp16 copy of W its scale.
__global__ void __launch_bounds__(256) head_exact_kernel(const HeadExact x, unsigned token_blocks, const HeadCopyW w_copy) {
  after_previous();
  if (blockIdx.x >= token_blocks) {
    rescale_w(w_copy, static_cast<int64_t>(blockIdx.x - token_blocks) * 256 + threadIdx.x,
              static_cast<int64_t>(gridDim.x - token_blocks) * 256);
    return;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= x.T) return;
  const float4 ri = x.en.row[t];
  if (ri.w == 0.f) return;
  __half* row = x.G + t * x.ld;            // of ids from v0
  const int begin = x.en.first[x.v0 / kHeadSplit * x.T + t];
  const int end = x.en.first[(x.v0 + x.n + kHeadSplit - 1) / kHeadSplit * x.T + t];
  exact_entries<true>(
      x.en.e + t * x.en.Ntot, begin, end, ri, static_cast<const char*>(x.h) + t * x.D * 2, x.W, x.D, threadIdx.x & 31,
      [&](int id, float sum) { return __half2float(row[id - x.v0]) - sum; },
      [&](int id, float v, bool heavy) {
        if (heavy) row[id - x.v0] = __float2half_rn(fabsf(v) > 65504.f ? copysignf(65504.f, v) : v);
      });
}

// ------------------------------------------------------------------ merge of partial statistics
__device__ __forceinline__ void warp_merge(float& m, float& z, float& u) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(kFull, m, o), z2 = __shfl_xor_sync(kFull, z, o), u2 = __shfl_xor_sync(kFull, u, o);
    // the lower lane's part first on both sides, so that all lanes hold the same bits
    if (threadIdx.x & o) {
      float a = m2, b = z2, c = u2;
      merge_part(a, b, c, m, z, u);
      m = a;
      z = b;
      u = c;
    } else {
      merge_part(m, z, u, m2, z2, u2);
    }
  }
}

__device__ __forceinline__ float entry_logit(const HeadFinish& f, int64_t t, int tot, int j, int id) {
  return f.picked != nullptr ? f.picked[t * tot + j] : f.logits[t * f.ld + id];
}

// A 64-bit logit likewise.
__device__ __forceinline__ float fine_base2(double l, float m) {
  return static_cast<float>(fma(l, 1.4426950408889634, -static_cast<double>(m)));
}

// The token's own numbers, entry k * 32 + lane of a warp's: the given tokens, or the teacher's and then the target.
struct Given {
  int id[kPerLane];
  bool there[kPerLane];
  float d[kPerLane];               // logits to base 2, over the row's reference
  bool bad, out;                   // an id, the target outside the vocabulary (then no logit was picked)
};

// ids: the token's; fine: their logits in 64 bits, or NULL.
__device__ __forceinline__ Given load_given(const HeadFinish& f, int64_t t, int lane, float m, const int* ids,
                                            const double* fine) {
  Given g;
  const int tot = f.N + (f.y != nullptr ? 1 : 0);
  const int y = f.y != nullptr ? f.y[t] : 0;
  g.bad = false;
  g.out = f.y != nullptr && (y < 0 || y >= f.V);
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    const int j = k * 32 + lane;
    g.id[k] = j < f.N ? ids[j] : j < tot ? y : -1;
    g.there[k] = g.id[k] >= 0 && g.id[k] < f.V;
    g.bad |= j < f.N && !g.there[k] && g.id[k] != -1;
    g.d[k] = 0.f;
    if (g.there[k] && !g.out)
      g.d[k] = fine != nullptr ? fine_base2(fine[j], m) : to_base2(entry_logit(f, t, tot, j, g.id[k]), f.log2e, m);
  }
  return g;
}

// The entries that hold more than 2^-4 of their row (at most 16 of them): their logits from products in 64 bits, and
// their terms of z and u with them.  The gradient of such an entry is a small difference, q less its coefficient, and
// is formed from these products too (head_exact.cuh), so it agrees with the log-sum-exp to fp32 rounding, whichever
// kernel made that of whatever batch.
template <bool BF16>
__device__ __forceinline__ void refine_given(const HeadFinish& f, int64_t t, int lane, float m, float& z, float& u,
                                             Given& g) {
  const float least = log2f(z) - 4.f;
  const char* h = static_cast<const char*>(f.h) + t * f.D * (BF16 ? 2 : 4);
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    unsigned todo = __ballot_sync(kFull, g.there[k] && !g.out && g.d[k] > least);
    while (todo != 0) {
      const int src = __ffs(todo) - 1;
      const int id[1] = {__shfl_sync(kFull, g.id[k], src)};
      const float was = __shfl_sync(kFull, g.d[k], src);
      bool before = false;                                 // named already: its terms are replaced
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) before |= i < k && g.id[i] == id[0];
      todo &= ~__ballot_sync(kFull, g.id[k] == id[0]);
      if (__any_sync(kFull, before)) continue;
      double l[1];
      dots64<BF16, 1>(h, f.W, f.D, id, lane, l);
      const float is = fine_base2(l[0], m);
      const float e0 = ex2(was), e1 = ex2(is);
      if (fabsf(m) < kLarge) {         // else m stands for a logit (low_base2), and their logits have few bits after the point
        z += e1 - e0;
        u += is * e1 - was * e0;
      }
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (g.id[i] == id[0]) g.d[i] = is;
    }
  }
}

// The token's outputs that need only the statistics, by one warp.  A log
// probability is ln 2 ((l log2(e) - m) - log2 z): both are small where it is,
// lse is not.
__device__ __forceinline__ void finish_token(const HeadFinish& f, int64_t t, int lane, float m, float logz, float mean,
                                             const Given& g) {
  // rounded once: the backward pass takes every q of the row from it
  if (lane == 0) f.stats[t] = static_cast<float>(0.6931471805599453 * (static_cast<double>(m) + static_cast<double>(logz)));
  bool bad = g.bad;
  if (f.y == nullptr) {
    if (lane == 0) f.stats[f.ldT + t] = kLn2 * (logz - mean);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
      if (k * 32 + lane < f.N) f.logp[t * f.N + k * 32 + lane] = g.there[k] ? kLn2 * (g.d[k] - logz) : 0.f;
  } else {
    const float w = f.weights != nullptr ? f.weights[t] : 1.f;
    bad |= g.out && w != 0.f;
    float z[kPerLane], top = -INFINITY, dy = 0.f;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int j = k * 32 + lane;
      z[k] = j < f.N && g.there[k] ? f.teacher[t * f.N + j] : -INFINITY;
      top = fmaxf(top, z[k]);
      if (j == f.N) dy = g.d[k];
    }
    top = warp_max(top);
    dy = __shfl_sync(kFull, dy, f.N & 31);
    const bool some = top > -INFINITY;
    float sum = 0.f, kd = 0.f;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      if (!some || g.out || k * 32 + lane >= f.N || !g.there[k]) continue;
      const float p = expf(z[k] - top);
      sum += p;
      if (p != 0.f) kd = fmaf(p, logz - g.d[k], kd);
    }
    sum = warp_sum(sum);
    kd = warp_sum(kd);
    kd = some && !g.out ? kLn2 * (kd / sum) : 0.f;
    if (lane == 0) {
      const float ce = g.out ? 0.f : kLn2 * (logz - dy);
      f.stats[f.ldT + t] = ce;
      f.stats[2 * f.ldT + t] = kd;
      const bool counts = !g.out && w != 0.f;  // 0 times a term that is not a number is not 0
      const float wce = counts ? w * ce : 0.f, wkd = counts ? w * kd : 0.f;
      f.terms[t] = wce;
      f.terms[f.ldT + t] = wkd;
      f.terms[2 * f.ldT + t] = fmaf(f.alpha, wkd, (1.f - f.alpha) * wce);
    }
  }
  if (__any_sync(kFull, bad) && lane == 0) set_flag(f.status, MLS_DEVFLAG_BAD_ID);
}

// A token from its row's merged statistics.
template <bool BF16>
__device__ __forceinline__ void finish_merged(const HeadFinish& f, int64_t t, int lane, float m, float z, float u) {
  Given g = load_given(f, t, lane, m, f.ids + t * f.N, nullptr);
  refine_given<BF16>(f, t, lane, m, z, u, g);
  finish_token(f, t, lane, m, log2f(z), u / z, g);
}

__global__ void __launch_bounds__(256) head_finish_kernel(const HeadFinish f) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= f.T) return;
  float m = -INFINITY, z = 0.f, u = 0.f;
  for (int s = lane; s < f.n_splits; s += 32) {
    const HeadPart p = f.part[t * f.n_splits + s];
    merge_part(m, z, u, p.x, p.y, p.z);
  }
  warp_merge(m, z, u);
  finish_merged<true>(f, t, lane, m, z, u);
}

// The same for the few tokens of one block, and the means of their loss terms:
// one launch in place of two.

__global__ void __launch_bounds__(1024) head_finish_loss_kernel(const HeadFinish f) {
  after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t t = warp; t < f.T; t += 32) {
    float m = -INFINITY, z = 0.f, u = 0.f;
    for (int s = lane; s < f.n_splits; s += 32) {
      const HeadPart p = f.part[t * f.n_splits + s];
      merge_part(m, z, u, p.x, p.y, p.z);
    }
    warp_merge(m, z, u);
    finish_merged<true>(f, t, lane, m, z, u);
  }
  __syncthreads();
  if (warp < 3) {
    float sum = 0.f;
    for (int64_t t = lane; t < f.T; t += 32) sum += f.terms[warp * f.ldT + t];
    sum = warp_sum(sum);
    if (lane == 0) f.losses[warp] = sum / static_cast<float>(f.T);
  }
}

// The same from the logits of a whole row (fp32 path without alternatives), one
// block per token: one launch in place of the splits' statistics and their merge.
__global__ void __launch_bounds__(256) head_finish_rows_kernel(const HeadFinish f) {
  __shared__ float sm[8], sz[8], su[8];
  after_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const float* row = f.logits + t * f.ld;
  float top = -INFINITY;
  for (int v = threadIdx.x; v < f.V; v += 256) top = fmaxf(top, row[v]);
  top = warp_max(top);
  if (lane == 0) sm[warp] = top;
  __syncthreads();
  top = warp_max(lane < 8 ? sm[lane] : -INFINITY);
  const bool large = fabsf(top) > kLarge;
  const float low = fmaxf(top, kLowest), m = (large ? low : top) * f.log2e;
  float z = 0.f, u = 0.f;
  for (int v = threadIdx.x; v < f.V; v += 256) {
    const float d = large ? low_base2(row[v], f.log2e, low) : max_nan(to_base2(row[v], f.log2e, m), -200.f), e = ex2(d);
    z += e;
    u = fmaf(d, e, u);
  }
  z = warp_sum(z);
  u = warp_sum(u);
  if (lane == 0) {
    sz[warp] = z;
    su[warp] = u;
  }
  __syncthreads();
  if (warp != 0) return;
  z = warp_sum(lane < 8 ? sz[lane] : 0.f);
  u = warp_sum(lane < 8 ? su[lane] : 0.f);
  finish_merged<false>(f, t, lane, m, z, u);
}

// ------------------------------------------------------------------ top alternatives
// One block per token.  The C = min(V, K + 4) largest logits by (value
// descending, id ascending) lie in the C splits with the largest maxima by
// (maximum descending, split ascending): were one of them in another split,
// each chosen split's first maximum would come before it.  So only those
// splits' logits are read.  Which they are is decided to 1/16: the maxima are
// counted in 256 bins below the largest, the bin of the C-th is the border, and
// a logit past it can be dropped too.  What is left (a few more than C) is
// ranked by counting.  Where the border is past the bins or too much is left
// (equal logits), radix selection over the whole row takes the place of it.
// A logit that is not a number is passed over everywhere (its key, where it has
// one, lies below that of -infinity).
//
// The candidates are then ranked by their products again, so that the ids do
// not depend on the tile a token fell into.  First with fp32 sums of 8
// products, added in 64 bits: each such sum is off by at most 7 half units of
// sum |h_i w_i|, a whole product by 7 2^-24 |h| |w| (Cauchy-Schwarz).  Where two
// neighbours among the first K + 1 are nearer than twice that, the token's
// candidates are multiplied once more with every product exact and added in 64
// bits; then only equal logits tie, and the lower id comes first.
//
// That is the order of all logits if none that was left out can reach the K-th:
// the last candidate's fp32 logit, and so every one left out, lies below the
// K-th's product by more than an fp32 logit can be off.  Four candidates more
// than K make that so for nearly every row (K = 32 of 49152 columns at D = 2304:
// a bound of 0.004 for logits that spread by 2, the gap of four places 0.06).
// Elsewhere (rows of W that differ in their last bits) every logit that can
// reach it, up to kWide of them, is multiplied exactly and ranked.
//
// The candidates' terms of z and u, the ones that weigh, are replaced by those
// of these products, which are more exact than the tensor cores' sums, and so
// are the given tokens' logits.
//
// The selection is a chain of short dependent steps (a block takes about 8 us
// for a token whatever the sizes), several blocks per SM hide each other's; the
// products read the rows of W that the candidates name (T = 4096, K = 32,
// D = 2304: 0.7 GB).  Selection and products in two kernels took 65 + 185 us
// there, in one 240: the one's steps hide behind the other's reads.
__device__ __forceinline__ uint32_t ordered(float f) {
  f += 0.f;                                              // -0 ranks as 0
  const uint32_t u = __float_as_uint(f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ uint64_t top_key(float v, uint32_t index) {
  return static_cast<uint64_t>(ordered(v)) << 32 | ~index;
}

// The k-th largest of n distinct keys (1 <= k <= n) as a lower bound: exactly k
// keys are at or above the returned value.  All kTopThreads threads of the block call it.
// keys: an array or a function of the index.
template <int kTopThreads, typename Keys>
__device__ uint64_t select_kth(const Keys& keys, int n, int k, int* hist, int* chosen) {
  const auto key_at = [&](int i) -> uint64_t {
    if constexpr (std::is_pointer_v<Keys>) return keys[i]; else return keys(i);
  };
  uint64_t prefix = 0;
  int shift = 56;
  for (; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kTopThreads) hist[i] = 0;
    __syncthreads();
    const uint64_t above = shift == 56 ? 0 : ~uint64_t(0) << (shift + 8);
    for (int i = threadIdx.x; i < n; i += kTopThreads) {
      const uint64_t key = key_at(i);
      if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // bins from the top, eight per lane: which bin holds the k-th, and how many lie above it
      const int lane = threadIdx.x;
      int own[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        own[i] = hist[255 - (lane * 8 + i)];
        sum += own[i];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < k && k <= before + own[i]) {
          chosen[0] = 255 - (lane * 8 + i);
          chosen[1] = k - before;
          chosen[2] = own[i];
        }
        before += own[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint64_t>(chosen[0]) << shift;
    k = chosen[1];
    const bool whole = chosen[2] == k;
    __syncthreads();
    if (whole) break;                                    // the whole bin is taken
  }
  return prefix;
}

// Products as dots64's with fp32 sums of 8 of them, and the squared norms of the rows.
template <int G>
__device__ __forceinline__ void dots_fast(const void* h, const void* W, int64_t D, const int* id, int lane,
                                          double (&acc)[G], float (&w2)[G]) {
  const uint4* a = static_cast<const uint4*>(h);
  const uint4* b[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    acc[g] = 0.0;
    w2[g] = 0.f;
    b[g] = static_cast<const uint4*>(W) + id[g] * (D / 8);
  }
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
      float y[8], p = 0.f;
      bf16x8_to_f32(w[g], y);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        p = fmaf(x[k], y[k], p);
        w2[g] = fmaf(y[k], y[k], w2[g]);
      }
      acc[g] += static_cast<double>(p);
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[g] += __shfl_xor_sync(kFull, acc[g], o);
    w2[g] = warp_sum(w2[g]);
  }
}

// The fast form by the block's warps; the largest squared norm to *norm (as bits).
template <int G>
__device__ __forceinline__ void block_dots_fast(const void* h, const void* W, int64_t D, const int* id, int n,
                                                double* val, unsigned int* norm, int warp, int warps, int lane) {
  for (int i = warp * G; i < n; i += warps * G) {
    int own[G];
#pragma unroll
    for (int g = 0; g < G; ++g) own[g] = id[i + g < n ? i + g : n - 1];
    double acc[G];
    float w2[G];
    dots_fast<G>(h, W, D, own, lane, acc, w2);
    if (lane == 0) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (i + g < n) {
          val[i + g] = acc[g];
          atomicMax(norm, __float_as_uint(w2[g]));
        }
    }
  }
}

// val[i] = h . W[id[i]] for i < n, by the block's warps; norm (fp32 inputs, may be NULL): as above.
template <bool BF16, int G>
__device__ __forceinline__ void block_dots(const void* h, const void* W, int64_t D, const int* id, int n, double* val,
                                           int warp, int warps, int lane, unsigned int* norm = nullptr) {
  for (int i = warp * G; i < n; i += warps * G) {
    int own[G];
#pragma unroll
    for (int g = 0; g < G; ++g) own[g] = id[i + g < n ? i + g : n - 1];
    double acc[G];
    float w2[G];
    dots64<BF16, G>(h, W, D, own, lane, acc, norm != nullptr ? w2 : nullptr);
    if (lane == 0) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (i + g < n) {
          val[i + g] = acc[g];
          if (norm != nullptr) atomicMax(norm, __float_as_uint(w2[g]));
        }
    }
  }
}

constexpr int kBins = 256;
constexpr int kTopList = 1024;             // logits that the selection may leave, as keys
constexpr int kWide = 640;                 // logits about the K-th that are ranked exactly, in the same memory
static_assert(kWide * (sizeof(double) + sizeof(int)) <= kTopList * sizeof(uint64_t), "room");
constexpr int kTopSmemLimit = 200 * 1024;

struct TopSmem {
  int hist[kBins];
  int chosen[4];
  float part[32][2];                         // sums z and u of each warp's splits
  float h2;
  unsigned int w2;                           // largest squared norm of a candidate's row, as bits
  double kth;                                // product of the K-th, where the candidates were ranked again
  int count, n_sel, border;
  int given[kMaxEntries];                    // the given tokens' ids
  int id[2 * kMaxEntries + kTopMore];        // rows to multiply: the given tokens, then the candidates by rank
  double fine[2 * kMaxEntries + kTopMore];   // their products
  float tile[kMaxEntries + kTopMore];        // the candidates' fp32 logits, by rank
  int rank[kMaxEntries + kTopMore];          // their final ranks
  float dz[kMaxEntries + kTopMore], du[kMaxEntries + kTopMore];   // by final rank: a fixed order of summation
};

// The bin of a logit or maximum: 0 at the largest, one more per 1/16 below it.
__device__ __forceinline__ int bin_of(float largest, float v) {
  return min(kBins - 1, static_cast<int>((largest - v) * 16.f));
}

template <bool BF16, int kTopThreads>
__global__ void __launch_bounds__(kTopThreads) head_top_kernel(const HeadFinish f, int C) {
  constexpr int kWarps = kTopThreads / 32;
  extern __shared__ __align__(16) uint8_t raw[];
  TopSmem& s = *reinterpret_cast<TopSmem*>(raw);
  uint64_t* keys = reinterpret_cast<uint64_t*>(raw + (sizeof(TopSmem) + 15) / 16 * 16);   // [kTopList]
  float* maxima = reinterpret_cast<float*>(keys + kTopList);                              // [n_splits]
  int* sel = reinterpret_cast<int*>(maxima + f.n_splits);                                 // [n_splits]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int n_splits = f.n_splits;

  after_previous();
  if (threadIdx.x < f.N) {
    const int id = f.ids[t * f.N + threadIdx.x];
    s.given[threadIdx.x] = id;
    s.id[threadIdx.x] = id >= 0 && id < f.V ? id : 0;
  }
  for (int i = threadIdx.x; i < kBins; i += kTopThreads) s.hist[i] = 0;
  if (threadIdx.x == 0) {
    s.count = s.n_sel = 0;
    s.w2 = 0;
  }
  // the statistics, and the largest logit
  float m = -INFINITY, z = 0.f, u = 0.f, largest = -INFINITY;
  for (int i = threadIdx.x; i < n_splits; i += kTopThreads) {
    const HeadPart p = f.part[t * n_splits + i];
    maxima[i] = p.w;
    largest = fmaxf(largest, p.w);
    merge_part(m, z, u, p.x, p.y, p.z);
  }
  largest = warp_max(largest);
  if (lane == 0) s.dz[warp] = largest;
  __syncthreads();
  largest = warp_max(lane < kWarps ? s.dz[lane] : -INFINITY);
  {
    // one reference for the block: that of the split with the largest logit
    const float ref = fmaxf(largest, kLowest) * f.log2e;
    if (z > 0.f || z != z) {
      const float d = m - ref, e = ex2(d);
      u = e > 0.f ? e * fmaf(d, z, u) : 0.f;
      z *= e;
    }
    m = ref;
    z = warp_sum(z);
    u = warp_sum(u);
    if (lane == 0) {
      s.part[warp][0] = z;
      s.part[warp][1] = u;
    }
  }

  // the border bin of the maxima, the splits on this side of it, their logits on this side of it
  // (with fewer splits than candidates, the border of the logits themselves)
  const float* row = f.logits + t * f.ld;
  if (n_splits >= C) {
    for (int i = threadIdx.x; i < n_splits; i += kTopThreads) atomicAdd(&s.hist[bin_of(largest, maxima[i])], 1);
  } else {
    for (int i = threadIdx.x; i < f.V; i += kTopThreads)
      if (row[i] == row[i]) atomicAdd(&s.hist[bin_of(largest, row[i])], 1);
  }
  __syncthreads();
  if (warp == 0) {
    int own[kBins / 32], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / 32; ++i) {
      own[i] = s.hist[lane * (kBins / 32) + i];
      sum += own[i];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, before, o);
      if (lane >= o) before += v;
    }
    before -= sum;
    int border = kBins - 1;
#pragma unroll
    for (int i = kBins / 32 - 1; i >= 0; --i) {
      sum -= own[i];
      if (before + sum < C && C <= before + sum + own[i]) border = lane * (kBins / 32) + i;
    }
    border = __reduce_min_sync(kFull, border);
    if (lane == 0) s.border = border;
  }
  __syncthreads();
  const int border = s.border;
  for (int i = threadIdx.x; i < n_splits; i += kTopThreads)
    if (bin_of(largest, maxima[i]) <= border) sel[atomicAdd(&s.n_sel, 1)] = i;
  __syncthreads();
  const int n_take = s.n_sel;
  for (int i = warp; i < n_take; i += kWarps) {
    const int col = sel[i] * kHeadSplit + lane * 4;
    if (col >= f.V) continue;                            // rows are padded to a multiple of 64
    const float4 v4 = *reinterpret_cast<const float4*>(row + col);
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (col + k >= f.V || v[k] != v[k] || bin_of(largest, v[k]) > border) continue;
      const int at = atomicAdd(&s.count, 1);
      if (at < kTopList) keys[at] = top_key(v[k], static_cast<uint32_t>(col + k));
    }
  }
  __syncthreads();
  int n = s.count;
  if (n > kTopList) {
    // keys made from the logits on every pass; C of them are at or above the C-th
    const auto at = [&](int i) {
      const float v = row[i];
      return v == v ? top_key(v, static_cast<uint32_t>(i)) : static_cast<uint64_t>(~static_cast<uint32_t>(i));
    };
    const uint64_t last = select_kth<kTopThreads>(at, static_cast<int>(f.V), C, s.hist, s.chosen);
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < f.V; i += kTopThreads) {
      const uint64_t key = at(i);
      if (key >= last && key >> 32 != 0) keys[atomicAdd(&s.count, 1)] = key;
    }
    __syncthreads();
    n = s.count;
  }
  int have = n < C ? n : C;                              // fewer only where logits are not numbers
  for (int i = threadIdx.x; i < n; i += kTopThreads) {
    const uint64_t key = keys[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += keys[j] > key;
    if (rank < C) {
      s.id[f.N + rank] = static_cast<int>(~static_cast<uint32_t>(key));
      s.tile[rank] = unordered(static_cast<uint32_t>(key >> 32));
    }
  }
  __syncthreads();

  // the given tokens' and the candidates' logits as products
  const char* hrow = static_cast<const char*>(f.h) + t * f.D * (BF16 ? 2 : 4);
  const int items = f.N + have;
  if (warp == kWarps - 1) {
    // |h|^2, for the bounds on the sums' errors
    float h2 = 0.f;
    if constexpr (BF16) {
      for (int i = lane; i < f.D / 8; i += 32) {
        float x[8];
        bf16x8_to_f32(reinterpret_cast<const uint4*>(hrow)[i], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) h2 = fmaf(x[k], x[k], h2);
      }
    } else {
      for (int64_t i = lane; i < f.D; i += 32) {
        const float x = reinterpret_cast<const float*>(hrow)[i];
        h2 = fmaf(x, x, h2);
      }
    }
    h2 = warp_sum(h2);
    if (lane == 0) s.h2 = h2;
  }
  if constexpr (BF16) {
    if (items <= kWarps) block_dots_fast<1>(hrow, f.W, f.D, s.id, items, s.fine, &s.w2, warp, kWarps, lane);
    else if (items <= 3 * kWarps) block_dots_fast<3>(hrow, f.W, f.D, s.id, items, s.fine, &s.w2, warp, kWarps, lane);
    else block_dots_fast<5>(hrow, f.W, f.D, s.id, items, s.fine, &s.w2, warp, kWarps, lane);
  } else {
    block_dots<false, 3>(hrow, f.W, f.D, s.id, items, s.fine, warp, kWarps, lane, &s.w2);
  }
  __syncthreads();
  // still in that order, no two of the first K + 1 nearer than the error, none of the rest among the first K?
  const int r = threadIdx.x;
  const double* fine = s.fine + f.N;
  const float unit = 5.9604645e-8f * sqrtf(s.h2) * sqrtf(__uint_as_float(s.w2));   // 2^-24 of the largest |h| |w|
  bool keep = true;
  if ((r + 1 < have && r < f.K) || (r > f.K && r < have)) {
    double off = 0.0;                                    // fp32 inputs: these products are the exact ones
    if constexpr (BF16) off = 2.f * 8.f * unit;          // 7, and the norms' rounding
    keep = (r < f.K ? fine[r] - fine[r + 1] : fine[f.K - 1] - fine[r]) > off;
  }
  if (r < have) s.rank[r] = r;
  // doubles as ordered integers, so that every value (a NaN too) has one rank
  const auto order = [](double d) {
    const int64_t b = __double_as_longlong(d + 0.0);
    return b < 0 ? ~static_cast<uint64_t>(b) : static_cast<uint64_t>(b) | (uint64_t(1) << 63);
  };
  const bool again = __syncthreads_or(!keep);
  if (again) {
    if constexpr (BF16) block_dots<true, 3>(hrow, f.W, f.D, s.id + f.N, have, s.fine + f.N, warp, kWarps, lane);
    __syncthreads();
    if (r < have) {
      const uint64_t mine = order(fine[r]);
      int rank = 0;
      for (int i = 0; i < have; ++i) {
        const uint64_t other = order(fine[i]);
        rank += other > mine || (other == mine && s.id[f.N + i] < s.id[f.N + r]);
      }
      s.rank[r] = rank;
      if (rank == f.K - 1) s.kth = fine[r];
    }
    __syncthreads();
  }
  if (have == C && C < f.V) {
    // A logit of the row is off by at most D / 16 truncated sums (2^-23 of sum |h_i w_i| each; fp32: D rounded ones, half
    // of that each) and some 32 more, for rows of W up to twice as long as the candidates' longest.
    const double kth = again ? s.kth : fine[f.K - 1];
    const double least = kth - 4.0 * (static_cast<double>(f.D) * (BF16 ? 1.0 / 16 : 0.5) + 40.0) * unit;
    if (unit != 0.f && !(s.tile[C - 1] < least)) {
      double* val = reinterpret_cast<double*>(keys);     // [kWide]
      int* id = reinterpret_cast<int*>(val + kWide);     // [kWide]
      if (threadIdx.x == 0) s.count = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < f.V; i += kTopThreads) {
        const float v = row[i];
        if (v != v || v < least) continue;
        const int at = atomicAdd(&s.count, 1);
        if (at < kWide) id[at] = i;
      }
      __syncthreads();
      const int wide = s.count;
      if (wide <= kWide) {
        block_dots<BF16, 3>(hrow, f.W, f.D, id, wide, val, warp, kWarps, lane);
        __syncthreads();
        have = min(wide, C);
        for (int i = threadIdx.x; i < wide; i += kTopThreads) {
          const uint64_t mine = order(val[i]);
          int rank = 0;
          for (int j = 0; j < wide; ++j) {
            const uint64_t other = order(val[j]);
            rank += other > mine || (other == mine && id[j] < id[i]);
          }
          if (rank >= have) continue;
          s.id[f.N + rank] = id[i];
          s.fine[f.N + rank] = val[i];
          s.tile[rank] = row[id[i]];
          s.rank[rank] = rank;
        }
        __syncthreads();
      }
    }
  }
  const int rank = r < have ? s.rank[r] : 0;
  if (r < have) {
    const float was = to_base2(s.tile[r], f.log2e, m), is = fine_base2(fine[r], m);
    const float e0 = ex2(was), e1 = ex2(is);
    const bool fix = fabsf(m) < kLarge;
    s.dz[rank] = fix ? e1 - e0 : 0.f;
    s.du[rank] = fix ? (e1 > 0.f ? is * e1 : 0.f) - (e0 > 0.f ? was * e0 : 0.f) : 0.f;
  }
  __syncthreads();
  if (warp * 32 >= kMaxEntries + kTopMore) return;
  z = warp_sum(lane < kWarps ? s.part[lane][0] : 0.f);
  u = warp_sum(lane < kWarps ? s.part[lane][1] : 0.f);
  float dz = 0.f, du = 0.f;
  for (int i = lane; i < have; i += 32) {
    dz += s.dz[i];
    du += s.du[i];
  }
  dz = warp_sum(dz);
  du = warp_sum(du);
  z += dz;
  const float logz = log2f(z);
  if (warp == 0) finish_token(f, t, lane, m, logz, (u + du) / z, load_given(f, t, lane, m, s.given, s.fine));
  if (r < have && rank < f.K) {
    f.top_ids[t * f.K + rank] = s.id[f.N + r];
    f.top_logp[t * f.K + rank] = kLn2 * (fine_base2(fine[r], m) - logz);
  }
  if (r >= have && r < f.K) {
    f.top_ids[t * f.K + r] = -1;
    f.top_logp[t * f.K + r] = NAN;
  }
}

}  // namespace

size_t head_entries_bytes(int64_t T, int64_t V, int Ntot, bool backward) {
  size_t b = head_align(static_cast<size_t>(T) * Ntot * sizeof(int2));
  b += head_align(static_cast<size_t>(head_splits(V) + 1) * T);
  if (backward) b += head_align(static_cast<size_t>(T) * sizeof(float4)) + 256;
  return b;
}

HeadEntries head_entries_layout(int64_t T, int64_t V, int Ntot, bool backward, void* ws) {
  char* q = static_cast<char*>(ws);
  HeadEntries e{};
  e.Ntot = Ntot;
  e.e = reinterpret_cast<int2*>(q);
  q += head_align(static_cast<size_t>(T) * Ntot * sizeof(int2));
  e.first = reinterpret_cast<uint8_t*>(q);
  q += head_align(static_cast<size_t>(head_splits(V) + 1) * T);
  if (backward) {
    e.row = reinterpret_cast<float4*>(q);
    q += head_align(static_cast<size_t>(T) * sizeof(float4));
    e.smax = reinterpret_cast<unsigned int*>(q);
  }
  return e;
}

cudaError_t run_head_entries(const HeadEntriesIn& in, const HeadEntries& out, bool backward, int32_t* status,
                             const HeadCopyW* w, cudaStream_t st) {
  if (in.h != nullptr) {                                 // the maxima that scale the fp16 copies (bf16 backward)
    const cudaError_t err = cudaMemsetAsync(out.smax, 0, 2 * sizeof(unsigned int), st);
    if (err != cudaSuccess) return err;
  }
  const unsigned grid = static_cast<unsigned>((in.T + kEntryTokens - 1) / kEntryTokens);
  const unsigned more = w != nullptr ? head_copy_blocks(w->n_vec) : 0;
  return head_launch(head_entries_kernel, dim3(grid + more), 256, 0, st, in, out, backward,
                     static_cast<int>(head_splits(in.V)), grid, w != nullptr ? *w : HeadCopyW{}, status);
}

cudaError_t run_head_exact(const HeadExact& x, const HeadCopyW* w, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((x.T + 7) / 8);
  const unsigned more = w != nullptr ? head_copy_blocks(w->n_vec) : 0;
  return head_launch(head_exact_kernel, dim3(grid + more), 256, 0, st, x, grid, w != nullptr ? *w : HeadCopyW{});
}

cudaError_t run_head_finish(const HeadFinish& f, cudaStream_t st) {
  if (f.losses != nullptr) return head_launch(head_finish_loss_kernel, dim3(1), 1024, 0, st, f);
  if (f.part == nullptr) return head_launch(head_finish_rows_kernel, dim3(static_cast<unsigned>(f.T)), 256, 0, st, f);
  return head_launch(head_finish_kernel, dim3(static_cast<unsigned>((f.T + 7) / 8)), 256, 0, st, f);
}

cudaError_t run_head_top(const HeadFinish& f, cudaStream_t st) {
  const int C = static_cast<int>(f.V < f.K + kTopMore ? f.V : f.K + kTopMore);
  const size_t smem = (sizeof(TopSmem) + 15) / 16 * 16 + kTopList * sizeof(uint64_t) + static_cast<size_t>(f.n_splits) * 8;
  // Few tokens leave SMs idle: their blocks get the warps that help, one per product (T = 1, D = 2304, K = 8: the whole
  // call 50.2 us with 512 threads, 51.4 with 1024; T = 24, D = 1024, K = 20: 34.6 and 32.6).
  // Of many tokens small blocks are best, more of them in flight per SM, until the products outweigh the steps before
  // them (T = 4096, K = 32, with 128 and 256 threads: D = 64 103 and 120 us, 512 114 and 127, 2304 285 and 266).
  const bool few = f.all <= 148, short_list = C + f.N <= 16;
  const bool light = static_cast<int64_t>(C + f.N) * f.D <= 40000 || !f.bf16;
  const unsigned threads = few ? (short_list ? 512 : 1024) : light ? 128 : 256;
  auto fn = f.bf16 ? (threads == 1024  ? head_top_kernel<true, 1024>
                      : threads == 512 ? head_top_kernel<true, 512>
                      : threads == 256 ? head_top_kernel<true, 256>
                                       : head_top_kernel<true, 128>)
                   : (threads == 1024  ? head_top_kernel<false, 1024>
                      : threads == 512 ? head_top_kernel<false, 512>
                                       : head_top_kernel<false, 128>);
  // the limit is the same on every call: another host thread's call may set it between here and the launch
  const cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopSmemLimit);
  if (err != cudaSuccess) return err;
  return head_launch(fn, dim3(static_cast<unsigned>(f.T)), threads, smem, st, f, C);
}

}  // namespace mls
