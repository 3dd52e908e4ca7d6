// Logits of a few tokens (decoding steps), bf16: the head is read once, at the
// rate of memory, and nothing else matters.
//
// The roles of the operands are exchanged against the large tiles: 128 rows of
// W are the M side of tcgen05.mma and the tokens (padded to 16, 32, 64 or 128)
// its N side, so no tensor or TMEM row is spent on tokens that do not exist and
// a stage holds 16 KB of W for 2 to 16 KB of h.  One CTA per SM walks the
// 128-row tiles of W with all of its shared memory in flight.
//
// tcgen05.mma truncates as it accumulates; with few tokens there is TMEM to
// spare, so the K blocks go to several accumulators in turn that the epilogue
// adds in fp32: shorter runs, smaller error.
//
// The logits go to the workspace (T x V fp32, a small part of W's bytes) with
// the partial statistics of each 128 columns.  T = 1, V = 49152, D = 2304: 41 us,
// T = 24, D = 1024: 22 us (W at 5.9 TB/s after 5 to 7 us of start and tail; the
// large tiles took 62 and 29 us).
#include <cuda.h>

#include "head.h"
#include "head_dev.cuh"
#include "head_host.h"
#include "umma.cuh"

namespace mls {

namespace {

constexpr int kRows = 128;               // rows of W per tile: one split
constexpr int kBK = 64;
constexpr int kUK = 16;
constexpr int kThreads = 192;            // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
constexpr int kEpi = 128;

struct FewMaps {
  CUtensorMap w, h;
};

struct FewArgs {
  int T, V, kblocks, n_tiles;
  HeadPart* part;                  // [T][n_tiles]
  float* logits;                   // [T][ld]
  int64_t ld;
  float log2e;
  int32_t* status;
};

template <int TN>
struct Few {
  static constexpr int kAcc = head_few_parts(TN);                    // accumulators per buffer
  static constexpr int kCols = 2 * kAcc * TN;                        // TMEM columns: two buffers
  static constexpr int kPad = kRows + 4;
  static constexpr int kStageBytes = kRows * kBK * 2 + TN * kBK * 2;
  static constexpr int kFixed = TN * kPad * 4 + 2048;
  static constexpr int kStages = (225 * 1024 - kFixed) / kStageBytes;
};

template <int TN>
struct __align__(1024) FewSmem {
  uint8_t w[Few<TN>::kStages][kRows * kBK * 2];
  uint8_t h[Few<TN>::kStages][TN * kBK * 2];
  float stage[TN][Few<TN>::kPad];
  uint64_t full[Few<TN>::kStages];
  uint64_t empty[Few<TN>::kStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpi) : "memory"); }

template <int TN>
__global__ void __launch_bounds__(kThreads, 1) head_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  using F = Few<TN>;
  constexpr int kStages = F::kStages;
  extern __shared__ uint8_t smem_raw[];
  FewSmem<TN>& s = *reinterpret_cast<FewSmem<TN>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &s.abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kEpi / 32);
    }
    mbar_init(&s.drain, 1);
    s.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.h);
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_base, F::kCols);
    tmem_relinquish();
  }
  // The thread that made the barriers is the one that loads: its first loads are on their way before the other warps
  // are set up (the first tile's K blocks, as many as the ring holds).
  after_previous();
  const int early = static_cast<int>(blockIdx.x) < a.n_tiles ? (a.kblocks < kStages ? a.kblocks : kStages) : 0;
  if (threadIdx.x == 0) {
    for (int kb = 0; kb < early; ++kb) {
      mbar_arrive_expect_tx(&s.full[kb], F::kStageBytes);
      tma_load_2d(&maps.w, &s.full[kb], s.w[kb], kb * kBK, static_cast<int>(blockIdx.x) * kRows);
      tma_load_2d(&maps.h, &s.full[kb], s.h[kb], kb * kBK, 0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  const int n_acc = a.kblocks < F::kAcc ? a.kblocks : F::kAcc;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t stage = early % kStages, phase = early / kStages, issued = early;
      bool ok = true;
      for (int tile = blockIdx.x; tile < a.n_tiles && ok; tile += gridDim.x) {
        for (int kb = tile == static_cast<int>(blockIdx.x) ? early : 0; kb < a.kblocks; ++kb) {
          if (!mbar_wait(&s.empty[stage], phase ^ 1, abort, a.status)) { ok = false; break; }
          mbar_arrive_expect_tx(&s.full[stage], F::kStageBytes);
          tma_load_2d(&maps.w, &s.full[stage], s.w[stage], kb * kBK, tile * kRows);
          tma_load_2d(&maps.h, &s.full[stage], s.h[stage], kb * kBK, 0);
          ++issued;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        // let every load already issued land before the CTA can exit
        const uint32_t n = issued < kStages ? issued : kStages;
        for (uint32_t i = 0; i < n; ++i) {
          if (stage == 0) { stage = kStages - 1; phase ^= 1; } else { --stage; }
          int dummy = 0;
          (void)mbar_wait(&s.full[stage], phase, &dummy, a.status);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(kRows, TN, false, false);
      uint32_t stage = 0, phase = 0, iter = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < a.n_tiles && ok; tile += gridDim.x, ++iter) {
        const uint32_t buf = iter & 1;
        if (!mbar_wait(&s.tempty[buf], ((iter >> 1) & 1) ^ 1, abort, a.status)) break;
        tc_fence_after();
        const uint32_t base = tmem + buf * (F::kAcc * TN);
        for (int kb = 0; kb < a.kblocks; ++kb) {
          if (!mbar_wait(&s.full[stage], phase, abort, a.status)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(smem_u32(s.w[stage]), 16, 1024);
          const uint64_t db = smem_desc_sw128(smem_u32(s.h[stage]), 16, 1024);
          const uint32_t d = base + (kb % F::kAcc) * TN;
#pragma unroll
          for (int k = 0; k < kBK / kUK; ++k)
            umma_bf16(d, da + static_cast<uint64_t>(k * 2), db + static_cast<uint64_t>(k * 2), idesc,
                      kb >= F::kAcc || k > 0);
          umma_commit(&s.empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (ok) umma_commit(&s.tfull[buf]);
      }
      umma_commit(&s.drain);
      int dummy = 0;
      (void)mbar_wait(&s.drain, 0, &dummy, a.status);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int v_in = q * 32 + lane;                       // this thread's row of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    constexpr int kSub = kEpi / TN > 0 ? kEpi / TN : 1;   // threads per token in the statistics
    const int e = threadIdx.x - 64;
    uint32_t iter = 0;
    for (int tile = blockIdx.x; tile < a.n_tiles; tile += gridDim.x, ++iter) {
      const uint32_t buf = iter & 1;
      const bool ok = mbar_wait(&s.tfull[buf], (iter >> 1) & 1, abort, a.status);
      // every epilogue warp leaves together: they share the staging barrier
      int go;
      asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.red.and.pred q, 2, %2, p;\n\t"
                   "selp.s32 %0, 1, 0, q;\n\t}" : "=r"(go) : "r"(static_cast<int>(ok)), "n"(kEpi) : "memory");
      if (!go) break;
      tc_fence_after();
      const int v = tile * kRows + v_in;
#pragma unroll 1
      for (int c = 0; c < TN; c += 16) {
        float sum[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[k] = 0.f;
        for (int j = 0; j < n_acc; ++j) {
          float r[16];
          tmem_ld16(lane_base + buf * (F::kAcc * TN) + j * TN + c, r);
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[k] += r[k];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          s.stage[c + k][v_in] = sum[k];
          if (c + k < a.T && v < a.V) a.logits[(c + k) * a.ld + v] = sum[k];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.tempty[buf]);
      epi_sync();
      {
        const int t = e / kSub, sub = e % kSub;
        const int n = a.V - tile * kRows;                 // rows of the tile that exist
        // at most 32 values of the token in registers at a time, so that their loads do not wait for one another
        constexpr int kOwn = kRows / kSub, kChunk = kOwn < 32 ? kOwn : 32;
        float top = -INFINITY, m = -INFINITY, z = 0.f, u = 0.f;
#pragma unroll 1
        for (int c = 0; c < kOwn; c += kChunk) {
          float l[kChunk], cm = -INFINITY;
#pragma unroll
          for (int k = 0; k < kChunk; ++k) {
            const int i = (c + k) * kSub + sub;
            l[k] = t < a.T && i < n ? s.stage[t][i] : -1.0e38f;      // finite to base 2 too: 0 times it is 0
            cm = fmaxf(cm, l[k]);
          }
#pragma unroll
          for (int o = kSub / 2; o > 0; o >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, o));
          if (fabsf(cm) > kLarge) {                        // the same for the threads of a token
            const float low = fmaxf(cm, kLowest);
            float cz = 0.f, cu = 0.f;
#pragma unroll
            for (int k = 0; k < kChunk; ++k) {
              const float d = low_base2(l[k], a.log2e, low), x = ex2(d);
              cz += x;
              cu = fmaf(d, x, cu);
            }
            merge_part(m, z, u, low * a.log2e, cz, cu);
            top = fmaxf(top, cm);
          } else {
            if (cm > top) {
              const float next = cm * a.log2e;
              if (z > 0.f) {
                const float d = m - next, f = ex2(d);
                u = f > 0.f ? f * fmaf(d, z, u) : 0.f;
                z *= f;
              }
              top = cm;
              m = next;
            }
#pragma unroll
            for (int k = 0; k < kChunk; ++k) {
              const float d = max_nan(to_base2(l[k], a.log2e, m), -200.f), x = ex2(d);
              z += x;
              u = fmaf(d, x, u);
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int o = kSub / 2; o > 0; o >>= 1) {
          z += __shfl_xor_sync(0xffffffffu, z, o);
          u += __shfl_xor_sync(0xffffffffu, u, o);
        }
        if (t < a.T && sub == 0) a.part[static_cast<int64_t>(t) * a.n_tiles + tile] = make_float4(m, z, u, top);
      }
      epi_sync();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, F::kCols);
  }
}

template <int TN>
cudaError_t run_few(const FewMaps& maps, const FewArgs& a, cudaStream_t st) {
  static_assert(Few<TN>::kCols <= 512 && (Few<TN>::kCols & (Few<TN>::kCols - 1)) == 0, "TMEM columns");
  const size_t smem = sizeof(FewSmem<TN>) + 1024;
  static_assert(sizeof(FewSmem<TN>) + 1024 <= 227 * 1024, "shared memory");
  auto fn = head_few_kernel<TN>;
  const cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int sms = head_num_sms();
  return head_launch(fn, dim3(static_cast<unsigned>(a.n_tiles < sms ? a.n_tiles : sms)), kThreads, smem, st, maps, a);
}

}  // namespace

cudaError_t head_tc_few(const HeadProblem& p, const HeadForward& f, cudaStream_t st) {
  const int tn = head_few_width(f.T);
  FewMaps maps;
  if (!head_make_map(&maps.w, p.W, p.D, p.V, p.D, kBK, kRows, false)) return cudaErrorInvalidValue;
  if (!head_make_map(&maps.h, f.h, p.D, f.T, p.D, kBK, tn, false)) return cudaErrorInvalidValue;
  FewArgs a{};
  a.T = static_cast<int>(f.T);
  a.V = static_cast<int>(p.V);
  a.kblocks = static_cast<int>((p.D + kBK - 1) / kBK);
  a.n_tiles = static_cast<int>(head_splits(p.V));
  a.part = f.part;
  a.logits = f.logits;
  a.ld = f.ld;
  a.log2e = head_log2e(p.D, head_few_parts(tn));
  a.status = p.status;
  switch (tn) {
    case 16: return run_few<16>(maps, a, st);
    case 32: return run_few<32>(maps, a, st);
    case 64: return run_few<64>(maps, a, st);
    default: return run_few<128>(maps, a, st);
  }
}

}  // namespace mls
