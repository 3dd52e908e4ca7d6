// C ABI of the single-exit LM-head operators: argument checking, workspace
// layout and the order of the launches.  Every declaration, its meaning and its
// error behaviour is documented in include/mls.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "head.h"
#include "mls.h"

namespace {

using mls::head_align;
using mls::head_splits;
using mls::HeadEntries;
using mls::HeadEntriesIn;
using mls::HeadFinish;
using mls::HeadForward;
using mls::HeadPart;
using mls::HeadProblem;

// The workspace queries return the size that needs no split, or the largest
// split within this budget.
constexpr size_t kBudget = size_t(3) << 29;   // 1.5 GiB

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mls_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MLS_OK : MLS_ERR_CUDA; }

mls_status check_shape(int64_t T, int64_t D, int64_t V, mls_dtype dt) {
  if (T <= 0 || D <= 0 || V <= 0) return MLS_ERR_INVALID_ARG;
  if (dt != MLS_F32 && dt != MLS_BF16) return MLS_ERR_INVALID_ARG;
  // ids stay 1024 below 2^31 so that a tile's last column does not pass it
  if (T > INT_MAX - 1024 || V > INT_MAX - 1024 || D > 65536) return MLS_ERR_UNSUPPORTED;
  if (dt == MLS_BF16 && D % 64 != 0) return MLS_ERR_UNSUPPORTED;
  if (static_cast<double>(T) * static_cast<double>(V) >= 9.0e15) return MLS_ERR_UNSUPPORTED;
  return MLS_OK;
}

mls_status check_top(int64_t V, int K) {
  if (K < 0) return MLS_ERR_INVALID_ARG;
  if (K > mls::kMaxEntries || K > V) return MLS_ERR_UNSUPPORTED;
  if (K > 0 && V > (int64_t(1) << 21)) return MLS_ERR_UNSUPPORTED;   // the splits' maxima fit one block's shared memory
  return MLS_OK;
}

HeadProblem shape(int64_t T, int64_t D, int64_t V, mls_dtype dt) {
  HeadProblem p{};
  p.bf16 = dt == MLS_BF16;
  p.T = T;
  p.D = D;
  p.V = V;
  return p;
}

// Forward workspace: what every token has [entries, loss terms], then a block
// of Tb tokens' [partial statistics][picked logits][logits].
struct ForwardPlan {
  int64_t Tb, ld;
  bool store;                      // the logits are written (alternatives, few tokens, or fp32)
  size_t entries, terms, part, picked, logits;
  size_t total() const { return entries + terms + part + picked + logits; }
};

ForwardPlan forward_plan(const HeadProblem& p, int Ntot, int K, bool distill, int64_t Tb) {
  ForwardPlan f{};
  f.Tb = Tb;
  f.ld = (p.V + 63) / 64 * 64;
  f.store = K > 0 || !p.bf16 || p.T <= mls::kFewTokens;
  f.entries = f.store ? 0 : mls::head_entries_bytes(p.T, p.V, Ntot, false);
  f.terms = distill ? head_align(static_cast<size_t>(p.T) * 3 * sizeof(float)) : 0;
  f.part = head_align(static_cast<size_t>(Tb) * head_splits(p.V) * sizeof(HeadPart));
  f.picked = f.store ? 0 : head_align(static_cast<size_t>(Tb) * (Ntot > 0 ? Ntot : 1) * sizeof(float));
  f.logits = f.store ? head_align(static_cast<size_t>(Tb) * f.ld * sizeof(float)) : 0;
  return f;
}

constexpr int64_t kBlock = 256;    // tokens of a tile

// The largest block of tokens (all, or equal blocks of a multiple of 256) whose
// workspace fits in `budget`; the smallest block when none does.
ForwardPlan forward_fit(const HeadProblem& p, int Ntot, int K, bool distill, size_t budget) {
  ForwardPlan all = forward_plan(p, Ntot, K, distill, p.T);
  if (all.total() <= budget || p.T <= kBlock) return all;
  int64_t lo = 1, hi = (p.T + kBlock - 1) / kBlock;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (forward_plan(p, Ntot, K, distill, mid * kBlock).total() <= budget) lo = mid; else hi = mid - 1;
  }
  const int64_t n = (p.T + lo * kBlock - 1) / (lo * kBlock);
  const int64_t even = ((p.T + n - 1) / n + kBlock - 1) / kBlock * kBlock;
  return forward_plan(p, Ntot, K, distill, even < lo * kBlock ? even : lo * kBlock);
}

size_t forward_min(const HeadProblem& p, int Ntot, int K, bool distill) {
  return forward_plan(p, Ntot, K, distill, p.T < kBlock ? p.T : kBlock).total();
}

// Statistics, picks, alternatives and loss terms of every token; `f` holds the
// operator's own pointers.
cudaError_t forward(const HeadProblem& p, const HeadEntriesIn& in, int Ntot, HeadFinish f, const ForwardPlan& plan,
                    void* ws, cudaStream_t st) {
  char* q = static_cast<char*>(ws);
  cudaError_t err = cudaSuccess;
  HeadEntries en{};
  if (!plan.store) {
    en = mls::head_entries_layout(p.T, p.V, Ntot, false, q);
    err = mls::run_head_entries(in, en, false, p.status, nullptr, st);
    if (err != cudaSuccess) return err;
  }
  q += plan.entries;
  float* terms = reinterpret_cast<float*>(q);
  q += plan.terms;
  HeadPart* part = reinterpret_cast<HeadPart*>(q);
  q += plan.part;
  float* picked = reinterpret_cast<float*>(q);
  q += plan.picked;
  float* logits = plan.store ? reinterpret_cast<float*>(q) : nullptr;
  const size_t esize = p.bf16 ? 2 : 4;
  f.V = p.V;
  f.all = p.T;
  f.ldT = p.T;
  f.n_splits = static_cast<int>(head_splits(p.V));
  f.part = p.bf16 || f.K > 0 ? part : nullptr;
  f.log2e = !p.bf16 ? mls::head_log2e(0, 1)
            : p.T <= mls::kFewTokens ? mls::head_log2e(p.D, mls::head_few_parts(mls::head_few_width(p.T)))
                                     : mls::head_log2e(p.D, 1);
  f.logits = logits;
  f.ld = plan.ld;
  f.picked = plan.store ? nullptr : picked;
  f.bf16 = p.bf16;
  f.D = p.D;
  f.W = p.W;
  f.status = p.status;
  for (int64_t t0 = 0; t0 < p.T; t0 += plan.Tb) {
    const int64_t n = t0 + plan.Tb <= p.T ? plan.Tb : p.T - t0;
    const char* h = static_cast<const char*>(p.h) + t0 * p.D * esize;
    if (p.bf16) {
      HeadForward w{};
      w.T = n;
      w.h = h;
      w.part = part;
      w.logits = logits;
      w.ld = plan.ld;
      w.en = en;
      if (!plan.store) {
        w.en.e = en.e + t0 * Ntot;
        w.en.first = en.first + t0;
      }
      w.ld_first = p.T;
      w.picked = picked;
      err = p.T <= mls::kFewTokens ? mls::head_tc_few(p, w, st) : mls::head_tc_forward(p, w, st);
    } else {
      err = mls::head_simt_logits(p, t0, n, logits, plan.ld, f.K > 0 ? part : nullptr, st);
    }
    if (err != cudaSuccess) return err;
    HeadFinish b = f;
    b.T = n;
    b.h = h;
    b.ids = f.ids != nullptr ? f.ids + t0 * f.N : nullptr;
    b.logp = f.logp != nullptr ? f.logp + t0 * f.N : nullptr;
    b.stats = f.stats + t0;
    b.top_ids = f.top_ids != nullptr ? f.top_ids + t0 * f.K : nullptr;
    b.top_logp = f.top_logp != nullptr ? f.top_logp + t0 * f.K : nullptr;
    b.y = f.y != nullptr ? f.y + t0 : nullptr;
    b.teacher = f.teacher != nullptr ? f.teacher + t0 * f.N : nullptr;
    b.weights = f.weights != nullptr ? f.weights + t0 : nullptr;
    b.terms = terms + t0;
    err = f.K > 0 ? mls::run_head_top(b, st) : mls::run_head_finish(b, st);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// Backward workspace: [entries][bf16: a chunk's G' and copies; fp32: a block of tokens' logits].
int64_t simt_block(const HeadProblem& p, size_t budget) {
  const int64_t b = static_cast<int64_t>(budget / (static_cast<size_t>(p.V) * sizeof(float)));
  return b < 1 ? 1 : (b < p.T ? b : p.T);
}

size_t backward_min(const HeadProblem& p, int Ntot) {
  const size_t e = mls::head_entries_bytes(p.T, p.V, Ntot, true);
  if (!p.bf16) return e + head_align(static_cast<size_t>(simt_block(p, 0)) * p.V * sizeof(float));
  const size_t whole = mls::head_tc_bwd_bytes(p, p.V);
  if (p.V <= 256) return e + whole;
  const size_t one = mls::head_tc_bwd_bytes(p, 256);
  return e + (one < whole ? one : whole);
}

size_t backward_bytes(const HeadProblem& p, int Ntot) {
  const size_t e = mls::head_entries_bytes(p.T, p.V, Ntot, true);
  if (!p.bf16) return e + head_align(static_cast<size_t>(simt_block(p, kBudget)) * p.V * sizeof(float));
  // very many tokens: no chunk narrower than 4096 columns, whose dh sums would cost more than the products
  const int64_t least = p.V < 4096 ? p.V : 4096;
  int64_t Vc = mls::head_tc_bwd_chunk(p, kBudget);
  if (Vc < least) Vc = least;
  return e + mls::head_tc_bwd_bytes(p, Vc);
}

mls_status backward(const HeadProblem& p, HeadEntriesIn in, int Ntot, void* dh, void* dW, bool dW_bf16,
                    int accumulate, void* ws, size_t ws_bytes, cudaStream_t st) {
  const size_t e = mls::head_entries_bytes(p.T, p.V, Ntot, true);
  const HeadEntries en = mls::head_entries_layout(p.T, p.V, Ntot, true, ws);
  char* rest = static_cast<char*>(ws) + e;
  if (p.bf16) {
    in.h = p.h;
    in.D = p.D;
    const int64_t Vc = mls::head_tc_bwd_chunk(p, ws_bytes - e);
    if (Vc <= 0) return MLS_ERR_WORKSPACE;
    return from_cuda(mls::head_tc_backward(p, in, en, dh, dW, dW_bf16, accumulate, rest, Vc, st));
  }
  const cudaError_t err = mls::run_head_entries(in, en, true, p.status, nullptr, st);
  if (err != cudaSuccess) return MLS_ERR_CUDA;
  return from_cuda(mls::head_simt_backward(p, en, static_cast<float*>(dh), static_cast<float*>(dW), accumulate,
                                           reinterpret_cast<float*>(rest), simt_block(p, ws_bytes - e), st));
}

// 16-byte loads and stores, or single fp32 values on the CUDA-core path.
uintptr_t alignment(mls_dtype dt) { return dt == MLS_BF16 ? 16 : 4; }

mls_status check_backward(const void* dh, const void* dW, mls_dtype dt, mls_dtype dW_dt, int accumulate_dW) {
  if (dh == nullptr && dW == nullptr) return MLS_ERR_INVALID_ARG;
  if (!aligned(dh, alignment(dt)) || !aligned(dW, alignment(dt))) return MLS_ERR_UNSUPPORTED;
  if (dW != nullptr) {
    if (dW_dt != MLS_F32 && dW_dt != MLS_BF16) return MLS_ERR_INVALID_ARG;
    if (dW_dt == MLS_BF16 && dt != MLS_BF16) return MLS_ERR_UNSUPPORTED;
    // sums over steps are held in 32 bits
    if (dW_dt == MLS_BF16 && accumulate_dW != 0) return MLS_ERR_UNSUPPORTED;
  }
  return MLS_OK;
}

mls_status check_operands(const void* h, const void* W, mls_dtype dt) {
  if (h == nullptr || W == nullptr) return MLS_ERR_INVALID_ARG;
  return aligned(h, alignment(dt)) && aligned(W, alignment(dt)) ? MLS_OK : MLS_ERR_UNSUPPORTED;
}

mls_status check_workspace(const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need) return MLS_ERR_WORKSPACE;
  return aligned(ws, 16) ? MLS_OK : MLS_ERR_UNSUPPORTED;
}

}  // namespace

#define MLS_TRY(expr)                       \
  do {                                      \
    const mls_status mls_try_ = (expr);     \
    if (mls_try_ != MLS_OK) return mls_try_; \
  } while (0)

extern "C" {

mls_status mls_token_logprobs_workspace(int64_t T, int64_t D, int64_t V, int N, int K, mls_dtype dt, size_t* bytes,
                                        size_t* min_bytes) {
  if (bytes == nullptr || N < 0 || N + K < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  MLS_TRY(check_top(V, K));
  if (N > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  const HeadProblem p = shape(T, D, V, dt);
  *bytes = forward_fit(p, N, K, false, kBudget).total();
  if (min_bytes != nullptr) *min_bytes = forward_min(p, N, K, false);
  return MLS_OK;
}

mls_status mls_token_logprobs(int64_t T, int64_t D, int64_t V, int N, const int32_t* ids, const void* h, const void* W,
                              mls_dtype dt, float* logp, float* stats, int K, int32_t* top_ids, float* top_logp,
                              void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (N < 0 || N + K < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  MLS_TRY(check_top(V, K));
  if (N > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  MLS_TRY(check_operands(h, W, dt));
  if ((N > 0 && (ids == nullptr || logp == nullptr)) || stats == nullptr) return MLS_ERR_INVALID_ARG;
  if (K > 0 && (top_ids == nullptr || top_logp == nullptr)) return MLS_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(logp, 4) || !aligned(stats, 4) || !aligned(top_ids, 4) || !aligned(top_logp, 4))
    return MLS_ERR_UNSUPPORTED;
  HeadProblem p = shape(T, D, V, dt);
  p.h = h;
  p.W = W;
  p.status = dev_status;
  MLS_TRY(check_workspace(workspace, ws_bytes, forward_min(p, N, K, false)));
  MLS_TRY(mls::check_device());
  HeadEntriesIn in{};
  in.T = T;
  in.V = V;
  in.N = N;
  in.ids = ids;
  HeadFinish f{};
  f.N = N;
  f.ids = ids;
  f.logp = logp;
  f.stats = stats;
  f.K = K;
  f.top_ids = top_ids;
  f.top_logp = top_logp;
  return from_cuda(forward(p, in, N, f, forward_fit(p, N, K, false, ws_bytes), workspace,
                           static_cast<cudaStream_t>(stream)));
}

mls_status mls_token_logprobs_bwd_workspace(int64_t T, int64_t D, int64_t V, int N, mls_dtype dt, size_t* bytes,
                                            size_t* min_bytes) {
  if (bytes == nullptr || N < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  if (N > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  const HeadProblem p = shape(T, D, V, dt);
  *bytes = backward_bytes(p, N);
  if (min_bytes != nullptr) *min_bytes = backward_min(p, N);
  return MLS_OK;
}

mls_status mls_token_logprobs_bwd(int64_t T, int64_t D, int64_t V, int N, const int32_t* ids, const void* h,
                                  const void* W, mls_dtype dt, const float* stats, const float* g_logp,
                                  const float* g_entropy, void* dh, void* dW, mls_dtype dW_dt, int accumulate_dW,
                                  void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (N < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  if (N > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  MLS_TRY(check_operands(h, W, dt));
  if (ids == nullptr || stats == nullptr || g_logp == nullptr) return MLS_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(stats, 4) || !aligned(g_logp, 4) || !aligned(g_entropy, 4))
    return MLS_ERR_UNSUPPORTED;
  MLS_TRY(check_backward(dh, dW, dt, dW_dt, accumulate_dW));
  HeadProblem p = shape(T, D, V, dt);
  p.h = h;
  p.W = W;
  p.status = dev_status;
  MLS_TRY(check_workspace(workspace, ws_bytes, backward_min(p, N)));
  MLS_TRY(mls::check_device());
  HeadEntriesIn in{};
  in.T = T;
  in.V = V;
  in.N = N;
  in.ids = ids;
  in.stats = stats;
  in.g_logp = g_logp;
  in.g_entropy = g_entropy;
  return backward(p, in, N, dh, dW, dW_dt == MLS_BF16, accumulate_dW, workspace, ws_bytes,
                  static_cast<cudaStream_t>(stream));
}

mls_status mls_topk_distill_workspace(int64_t T, int64_t D, int64_t V, int K, mls_dtype dt, size_t* fwd_bytes,
                                      size_t* fwd_min, size_t* bwd_bytes, size_t* bwd_min) {
  if (fwd_bytes == nullptr || bwd_bytes == nullptr || K < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  if (K > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  const HeadProblem p = shape(T, D, V, dt);
  *fwd_bytes = forward_fit(p, K + 1, 0, true, kBudget).total();
  *bwd_bytes = backward_bytes(p, K + 1);
  if (fwd_min != nullptr) *fwd_min = forward_min(p, K + 1, 0, true);
  if (bwd_min != nullptr) *bwd_min = backward_min(p, K + 1);
  return MLS_OK;
}

mls_status mls_topk_distill_fwd(int64_t T, int64_t D, int64_t V, int K, const int32_t* y_targets,
                                const int32_t* teacher_ids, const float* teacher_logits, const float* token_weights,
                                const void* h, const void* W, float alpha_d, mls_dtype dt, float* losses, float* stats,
                                void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (K < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  if (K > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  MLS_TRY(check_operands(h, W, dt));
  if (y_targets == nullptr || teacher_ids == nullptr || teacher_logits == nullptr || losses == nullptr ||
      stats == nullptr || !std::isfinite(alpha_d))
    return MLS_ERR_INVALID_ARG;
  if (!aligned(y_targets, 4) || !aligned(teacher_ids, 4) || !aligned(teacher_logits, 4) ||
      !aligned(token_weights, 4) || !aligned(losses, 4) || !aligned(stats, 4))
    return MLS_ERR_UNSUPPORTED;
  HeadProblem p = shape(T, D, V, dt);
  p.h = h;
  p.W = W;
  p.status = dev_status;
  MLS_TRY(check_workspace(workspace, ws_bytes, forward_min(p, K + 1, 0, true)));
  MLS_TRY(mls::check_device());
  HeadEntriesIn in{};
  in.T = T;
  in.V = V;
  in.N = K;
  in.ids = teacher_ids;
  in.y = y_targets;
  in.teacher = teacher_logits;
  in.weights = token_weights;
  in.alpha = alpha_d;
  HeadFinish f{};
  f.N = K;
  f.ids = teacher_ids;
  f.stats = stats;
  f.y = y_targets;
  f.teacher = teacher_logits;
  f.weights = token_weights;
  f.alpha = alpha_d;
  const ForwardPlan plan = forward_fit(p, K + 1, 0, true, ws_bytes);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // as few tokens as a block has warps: one block finishes them and their means (90 tokens in one block took 4 us
  // more than two launches)
  const bool one = p.bf16 && T <= 32;
  f.losses = one ? losses : nullptr;
  MLS_TRY(from_cuda(forward(p, in, K + 1, f, plan, workspace, st)));
  if (one) return MLS_OK;
  const float* terms = reinterpret_cast<const float*>(static_cast<char*>(workspace) + plan.entries);
  return from_cuda(mls::launch_row_means(terms, 3, T, losses, st));
}

mls_status mls_topk_distill_bwd(int64_t T, int64_t D, int64_t V, int K, const int32_t* y_targets,
                                const int32_t* teacher_ids, const float* teacher_logits, const float* token_weights,
                                const void* h, const void* W, float alpha_d, mls_dtype dt, const float* stats,
                                float grad_scale, void* dh, void* dW, mls_dtype dW_dt, int accumulate_dW,
                                void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (K < 1) return MLS_ERR_INVALID_ARG;
  MLS_TRY(check_shape(T, D, V, dt));
  if (K > mls::kMaxEntries) return MLS_ERR_UNSUPPORTED;
  MLS_TRY(check_operands(h, W, dt));
  if (y_targets == nullptr || teacher_ids == nullptr || teacher_logits == nullptr || stats == nullptr ||
      !std::isfinite(alpha_d) || !std::isfinite(grad_scale))
    return MLS_ERR_INVALID_ARG;
  if (!aligned(y_targets, 4) || !aligned(teacher_ids, 4) || !aligned(teacher_logits, 4) ||
      !aligned(token_weights, 4) || !aligned(stats, 4))
    return MLS_ERR_UNSUPPORTED;
  MLS_TRY(check_backward(dh, dW, dt, dW_dt, accumulate_dW));
  HeadProblem p = shape(T, D, V, dt);
  p.h = h;
  p.W = W;
  p.status = dev_status;
  MLS_TRY(check_workspace(workspace, ws_bytes, backward_min(p, K + 1)));
  MLS_TRY(mls::check_device());
  HeadEntriesIn in{};
  in.T = T;
  in.V = V;
  in.N = K;
  in.ids = teacher_ids;
  in.stats = stats;
  in.y = y_targets;
  in.teacher = teacher_logits;
  in.weights = token_weights;
  in.alpha = alpha_d;
  in.grad = grad_scale / static_cast<float>(T);
  return backward(p, in, K + 1, dh, dW, dW_dt == MLS_BF16, accumulate_dW, workspace, ws_bytes,
                  static_cast<cudaStream_t>(stream));
}

}  // extern "C"
