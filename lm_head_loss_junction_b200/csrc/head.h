// Internal interface of the single-exit LM-head operators (log probabilities
// of given tokens; distillation from a teacher's top logits) between the
// C-ABI layer (head_api.cu), the tensor-core kernels (head_tc.cu), the
// per-token kernels (head_rows.cu) and the fp32 path (head_simt.cu).
//
// Both operators have the same logit gradient,
//   G[t, v] = s_t ( q[t, v] (A_t + B_t (l[t, v] - lse_t)) + sum over entries (v, c) of token t of c ),
// with q = softmax(l), a power of two s_t, and a short list of (id, coefficient)
// entries per token, so they share every kernel below the coefficients:
//   log probabilities: s A = -(sum g_n) - g_H H, s B = -g_H, entries (id_n, g_n)
//   distillation:      s A = w' ((1 - alpha) + alpha [any teacher token]), B = 0,
//                      entries (y, -w' (1 - alpha)), (id_k, -w' alpha p_k), w' = w grad_scale / T.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace mls {

constexpr int kHeadSplit = 128;      // vocabulary columns per partial statistic
constexpr int kMaxEntries = 64;      // given tokens, teacher tokens or alternatives per token
constexpr int kTopMore = 4;          // candidates beyond K that are ranked again in 64 bits

inline int64_t head_splits(int64_t V) { return (V + kHeadSplit - 1) / kHeadSplit; }
inline size_t head_align(size_t b) { return (b + 255) & ~size_t(255); }

// Partial softmax statistics of one token over one split, to base 2 (an
// exponential is then one fma and one instruction, and l log2(e) - m is rounded
// once): with a_v = l_v log2(e) - m for a reference m near the largest one,
// (m, z = sum 2^a, u = sum a 2^a, the largest logit itself).
typedef float4 HeadPart;

// log2(e) for logits of the tensor cores.  Each of the D / 16 steps of an
// accumulation truncates the running sum, which shrinks a logit: measured
// against 64 bits, by 0.20 to 0.28 x 2^-24 of itself per step for every D from
// 512 to 65536, logits of random rows, of a leant-to row and of heads with a mean
// row alike (0.26 to 0.27 from D = 8192 on).  A quarter of 2^-24 per step is given
// back here (D = 2304: the mean error of a logit falls from 2.1e-6 to under 0.2e-6
// of it, the root mean square from 4.8e-6 to 2.4e-6; plain fp32 sums have 0.9e-6.
// D = 65536, a leant-to row: 6.6e-5 to 0.6e-5).  A row whose sums are exact (a few
// entries, small whole numbers) was not shrunk and is off by what is given back,
// D 2^-30.  parts: accumulators that share the steps.
inline float head_log2e(int64_t D, int parts) {
  return static_cast<float>(1.4426950408889634 * (1.0 + static_cast<double>(D) / parts / 1073741824.0));
}

struct HeadProblem {
  bool bf16;
  int64_t T, D, V;
  const void* h;
  const void* W;
  int32_t* status;
};

// Where a token's own numbers come from.  N entries per token (ids [T][N]),
// plus the target y for the distillation (entry N).
struct HeadEntriesIn {
  int64_t T, V;
  int N;
  const void* h;                   // bf16 backward: [T][D], for its rows' largest magnitudes
  int64_t D;
  const int32_t* ids;              // [T][N]; -1: absent
  // log probabilities, backward
  const float* stats;              // [2][T]: lse, entropy (distillation: row 0 of [3][T])
  const float* g_logp;             // [T][N]
  const float* g_entropy;          // [T] or NULL
  // distillation
  const int32_t* y;                // [T], NULL for the log probabilities
  const float* teacher;            // [T][N] logits
  const float* weights;            // [T] or NULL (1)
  float alpha, grad;               // grad = grad_scale / T
};

// Entries sorted by id, and the first entry of every split: entries of token t
// in columns [128 s, 128 s + 128) are e[t][first[s][t]] .. e[t][first[s + 1][t]).
struct HeadEntries {
  int2* e;                         // [T][Ntot] (id, position or coefficient bits)
  uint8_t* first;                  // [splits + 1][T]
  float4* row;                     // [T] (lse, A, B, s); backward only
  unsigned int* smax;              // backward only, as float bits, set to 0 with the entries: [0] a bound on s_t |h_ti|
                                   // (a power of two), [1] the largest magnitude of the chunk of W
  int Ntot;
};
size_t head_entries_bytes(int64_t T, int64_t V, int Ntot, bool backward);
HeadEntries head_entries_layout(int64_t T, int64_t V, int Ntot, bool backward, void* ws);

// fp16 copies of bf16 operands for the gradient products (head_copy.cuh).
struct HeadCopyW {
  const void* src;
  __half* dst;
  int64_t n_vec;                   // vectors of 8 values; 0: nothing to do
  unsigned int* maxbits;
  float* inv;                      // 1 / the copy's scale
};
struct HeadCopyH {
  const void* src;
  __half* dst;
  int64_t n_vec;
  int vec_per_row;
  const float4* row;
  const unsigned int* smax;
};

// w (may be NULL): a copy of W made by further blocks of the same launch.
cudaError_t run_head_entries(const HeadEntriesIn& in, const HeadEntries& out, bool backward, int32_t* status,
                             const HeadCopyW* w, cudaStream_t st);

// G' of a chunk of the vocabulary, whose entries of much weight are formed again
// from products in 64 bits (bf16; head_exact.cuh).
struct HeadExact {
  int64_t T, D;
  const void* h;
  const void* W;                   // the whole of it
  HeadEntries en;
  __half* G;                       // [T][ld], column 0 is id v0
  int64_t ld, v0, n;
};
// w (may be NULL): a copy of W that further blocks of the launch give its scale.
cudaError_t run_head_exact(const HeadExact& x, const HeadCopyW* w, cudaStream_t st);

// ------------------------------------------------------------------ per-token results
struct HeadFinish {
  int64_t T, V;                    // tokens of this launch
  int64_t all;                     // of the whole call (no result depends on the pieces)
  int64_t ldT;                     // row stride of the [*][T] outputs
  int n_splits;
  const HeadPart* part;            // [T][n_splits], or NULL: from the logits (run_head_finish)
  float log2e;                     // of the logits
  const float* logits;             // [T][ld] or NULL
  int64_t ld;
  const float* picked;             // [T][Ntot] or NULL (then read from logits)
  int N;
  const int32_t* ids;              // [T][N]
  float* logp;                     // [T][N]
  float* stats;                    // [2][ldT] or [3][ldT]
  // alternatives
  int K;
  int32_t* top_ids;                // [T][K]
  float* top_logp;                 // [T][K]
  bool bf16;
  int64_t D;
  const void* h;
  const void* W;
  // distillation
  const int32_t* y;
  const float* teacher;
  const float* weights;
  float alpha;
  float* terms;                    // [3][ldT]
  float* losses;                   // [3] means of the terms, or NULL: left to the caller (run_head_finish)
  int32_t* status;
};
cudaError_t run_head_finish(const HeadFinish& f, cudaStream_t st);      // lse, entropy, picks or loss terms
cudaError_t run_head_top(const HeadFinish& f, cudaStream_t st);         // the same and the alternatives (needs logits)

// ------------------------------------------------------------------ tensor-core path (bf16)
// Logits of tokens [0, T) in 256 x 256 tiles: partial statistics, and either
// the picked logits of the entries or (logits != NULL) the logits themselves.
struct HeadForward {
  int64_t T;                       // tokens of this launch
  const void* h;                   // its rows
  HeadPart* part;                  // [T][n_splits]
  float* logits;                   // [T][ld] or NULL
  int64_t ld;
  HeadEntries en;                  // entries of the launch's tokens (logits == NULL)
  int64_t ld_first;                // row stride of en.first
  float* picked;                   // [T][Ntot]
};
cudaError_t head_tc_forward(const HeadProblem& p, const HeadForward& f, cudaStream_t st);

// The same for at most kFewTokens tokens, logits always written (f.logits != NULL).
constexpr int64_t kFewTokens = 128;
inline int head_few_width(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }
constexpr int head_few_parts(int width) { return width <= 32 ? 8 : 256 / width; }
cudaError_t head_tc_few(const HeadProblem& p, const HeadForward& f, cudaStream_t st);

// dh and dW (either may be NULL) from the entries, which it makes first, one
// chunk of the vocabulary at a time.
size_t head_tc_bwd_bytes(const HeadProblem& p, int64_t Vc);
int64_t head_tc_bwd_chunk(const HeadProblem& p, size_t budget);
cudaError_t head_tc_backward(const HeadProblem& p, const HeadEntriesIn& in, const HeadEntries& en, void* dh, void* dW,
                             bool dW_bf16, int accumulate, void* ws, int64_t Vc, cudaStream_t st);

// ------------------------------------------------------------------ CUDA-core path (fp32)
cudaError_t head_simt_logits(const HeadProblem& p, int64_t t0, int64_t Tb, float* logits, int64_t ld,
                             HeadPart* part, cudaStream_t st);
cudaError_t head_simt_backward(const HeadProblem& p, const HeadEntries& en, float* dh, float* dW, int accumulate,
                               float* logits, int64_t Tb, cudaStream_t st);

}  // namespace mls
