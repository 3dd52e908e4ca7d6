// Tensor-core (tcgen05 + TMEM + TMA) kernels of the single-exit LM-head
// operators, bf16.
//
// One persistent kernel on CTA pairs computes 256 x 256 output tiles
// (tcgen05.mma.cta_group::2, each CTA holding 128 rows of A, half of B and its
// half of the fp32 accumulator in TMEM, two accumulator buffers) and differs
// in what the eight epilogue warps of each CTA do with the accumulator:
//   stats   logits h W^T of 256 tokens x 256 columns -> softmax statistics per
//           token and 128-column split (HeadPart), and the logits of the token's
//           entries; the logits themselves are not written
//   logits  the same statistics, and the logits in fp32 (for the alternatives)
//   grad    the logits again -> G' = q (A + B (l - lse)) + entries in fp16
//   dh      G' W (K = columns of the chunk), scaled per row
//   dw      G'^T h (K = tokens)
// All five are bound by the tensor pipe once T passes a few hundred tokens (dh
// and dw at 1.36 and 1.39 PFLOP/s, stats at 1.27, grad at 1.20 with T = 2048,
// D = 1024, V = 49152; in long runs by the power cap, within 4% of cuBLAS's
// products of the same shapes), and by reading W and a launch's own start and
// tail below that.
//
// G' is fp16 (11-bit significand), not bf16 (8): the few large entries of a
// peaked row dominate the gradient's error.  A row is stored divided by a
// power of two s_t that brings its bound to 2^14, so that rows of very
// different weight keep the same relative precision and the small
// probabilities of a peaked row keep theirs; dh multiplies by s_t in the
// epilogue and dw reads h rows that were multiplied by s_t when they were
// copied to fp16 (powers of two change no significand).
#include <cuda.h>
#include <cuda_fp16.h>
#include <atomic>
#include <mutex>

#include "head.h"
#include "head_copy.cuh"
#include "head_dev.cuh"
#include "head_host.h"
#include "umma.cuh"

namespace mls {

namespace {

constexpr int kBM = 128;                 // rows of A per CTA
constexpr int kBN = 256;                 // columns of a tile
constexpr int kBK = 64;                  // one 128-byte swizzle row of 16-bit values
constexpr int kUK = 16;                  // K per tcgen05.mma
constexpr int kStages = 6;               // 32 KB per stage and CTA
constexpr int kEpiWarps = 8;             // two per TMEM lane quadrant, 128 columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kCopyThreads = 64;         // two more warps: as many registers per thread as without them
constexpr int kStageRow = 80;            // bytes of a staged row of 32 fp16 (padded against bank conflicts)
constexpr int kStageWarp = 32 * 128;     // bytes of a warp's staging rows: 32 x 32 fp32, or fp16 rows
constexpr int kGroupM = 8;               // row tiles per raster group: they share their A panels in L2
constexpr float kMasked = -1.0e38f;      // logit of a column past V: finite to base 2 too, so that 0 times it is 0

enum Epi { kStats, kLogits, kGrad, kDh, kDw };

// W's copy in a kernel of its own (later chunks of few tokens).
__global__ void __launch_bounds__(256) head_copy_kernel(const HeadCopyW w) {
  after_previous();
  copy_w(w, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, static_cast<int64_t>(gridDim.x) * blockDim.x);
}

struct TileMaps {
  CUtensorMap a, b;
};

struct TileArgs {
  int rows, cols;                  // extents of the output
  int kblocks;
  int n_mt, n_nt;                  // tiles down and across
  int parts, part_kblocks;         // K in parts (dh only): each part's tiles are units of their own
  int units;
  // stats, logits, grad
  int v0;                          // vocabulary id of column 0
  float log2e;                     // of the logits
  int n_splits;                    // splits of a row of part
  HeadPart* part;
  float* logits;
  int64_t ld;                      // row stride of logits or G'
  const int2* e;
  const uint8_t* first;
  int64_t ld_first;
  int Ntot;
  float* picked;
  const float4* row;
  __half* G;
  int gcols;                       // columns of G' that are written (a multiple of 64)
  // dh, dw
  void* out;
  float* acc;                      // dh partial sums of earlier chunks [rows][cols] (NULL: none)
  int accumulate;
  const float* inv;                // dh, device: 1 / scale of the fp16 copy of W
  const unsigned int* smax;        // dw, device: the bound that scales the copy of h
  HeadCopyW copy_w;                // grad: fp16 copies made by two more warps
  HeadCopyH copy_h;
  int w_copied;                    // W's copy is made already, they give it its scale
  int32_t* status;
};

// What one turn of a CTA pair computes: a tile over kblocks [kb0, kb1).
struct Unit {
  int mt, nt, part, kb0, kb1;
};

struct __align__(1024) TileSmem {
  uint8_t a[kStages][kBM * kBK * 2];
  uint8_t b[kStages][(kBN / 2) * kBK * 2];
  uint8_t stage[kEpiWarps][kStageWarp];
  uint64_t full[kStages];          // leader: both CTAs' bytes
  uint64_t empty[kStages];
  uint64_t tfull[2];
  uint64_t tempty[2];              // leader: 16 epilogue warps
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  const bool ok = mbar_wait(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ Unit unit_at(const TileArgs& a, int i) {
  Unit u;
  const int tiles = a.n_mt * a.n_nt;
  u.part = i / tiles;
  i -= u.part * tiles;
  const int per_group = kGroupM * a.n_nt;
  const int g = i / per_group;
  const int first = g * kGroupM;
  const int gm = min(kGroupM, a.n_mt - first);
  const int r = i - g * per_group;
  u.nt = r / gm;
  u.mt = first + r % gm;
  u.kb0 = u.part * a.part_kblocks;
  u.kb1 = min(a.kblocks, u.kb0 + a.part_kblocks);
  return u;
}

__device__ __forceinline__ uint32_t pack_g2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Columns at or past `left` of a 32-column chunk do not exist.
__device__ __forceinline__ void mask_columns(float (&r)[32], int left) {
  if (left < 32) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k >= left) r[k] = kMasked;
  }
}

// The entries of one token inside its split, in ascending id order, two of
// them loaded ahead.
struct EntryWalk {
  const int2* p;
  int n;
  int2 cur, nxt;
  __device__ __forceinline__ int2 load() {
    if (n <= 0) return make_int2(INT32_MAX, 0);
    --n;
    return *p++;
  }
  __device__ __forceinline__ void start(const TileArgs& a, bool valid, int t, int split) {
    n = 0;
    if (valid) {
      const int b = a.first[static_cast<int64_t>(split) * a.ld_first + t];
      n = a.first[static_cast<int64_t>(split + 1) * a.ld_first + t] - b;
      p = a.e + static_cast<int64_t>(t) * a.Ntot + b;
    }
    cur = load();
    nxt = load();
  }
  __device__ __forceinline__ void next() {
    cur = nxt;
    nxt = load();
  }
};

// What a row of a tile needs besides its accumulator, loaded before the
// epilogue waits for the accumulator.  (Asking a whole tile ahead measured
// slower: 2.91 against 2.86 ms for the step at T = 8192, D = 1024, 64 entries.)
struct RowAhead {
  EntryWalk en;
  float4 ri;                       // (lse, A, B, s)
};

// A warp's 32 x 32 fp32 chunk in its staging rows: 16-byte pieces permuted by
// row, so that rows and columns of pieces are free of bank conflicts.
__device__ __forceinline__ float4* staged(uint8_t* stage, int row, int piece) {
  return reinterpret_cast<float4*>(stage + row * 128 + ((piece ^ (row & 7)) * 16));
}

__device__ __forceinline__ float* staged_at(uint8_t* stage, int row, int col) {
  return reinterpret_cast<float*>(staged(stage, row, col >> 2)) + (col & 3);
}

// This lane's row.  (Only a __syncwarp makes it visible to other lanes.)
__device__ __forceinline__ void stage_row(uint8_t* stage, int lane, const float (&r)[32]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) *staged(stage, lane, k) = make_float4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
}

// This lane's row of 32 values as 16-bit pairs through the staging rows (of 80
// bytes here), so that a store instruction writes 8 rows x 64 contiguous bytes:
// dst is this lane's piece (row lane / 4, 16 bytes lane % 4) of the chunk's
// first 8 rows, `left` the rows from there on that exist.
__device__ __forceinline__ void store_pairs(uint8_t* stage, int lane, const uint32_t (&w)[16], uint8_t* dst,
                                            int64_t row_bytes, int64_t left) {
  uint4* mine = reinterpret_cast<uint4*>(stage + lane * kStageRow);
#pragma unroll
  for (int k = 0; k < 4; ++k) mine[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  __syncwarp();
  const uint8_t* src = stage + (lane >> 2) * kStageRow + (lane & 3) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (8 * i < left)
      *reinterpret_cast<uint4*>(dst + 8 * i * row_bytes) = *reinterpret_cast<const uint4*>(src + 8 * i * kStageRow);
  __syncwarp();
}

// Tells the leader that an accumulator buffer was read.  Relaxed: what it orders
// are TMEM reads, which are complete (tcgen05.wait::ld) and fenced; a release
// would also wait for the epilogue's global stores to be acknowledged, about a
// microsecond per tile.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Two powers of two a and s as the factors of a s, each about its root: a sum
// times a alone, or a s itself, may be out of fp32's range where sum a s is not.
__device__ __forceinline__ void split_scale(float a, float s, float& f1, float& f2) {
  f1 = f2 = 0.f;
  if (!(s > 0.f)) return;
  const int e = ilogbf(a) + ilogbf(s), half = e / 2;
  f1 = ldexpf(1.f, half);
  f2 = ldexpf(1.f, e - half);
}

// A_MN / B_MN: the operand is stored with its M / N dimension contiguous
// (boxes of 64 x 64), otherwise with K contiguous.
template <Epi EPI>
struct Layout {
  static constexpr bool a_mn = EPI == kDw;
  static constexpr bool b_mn = EPI == kDh || EPI == kDw;
  static constexpr bool f16 = EPI == kDh || EPI == kDw;
};

template <Epi EPI, bool OUT_BF16>
__device__ __forceinline__ void epilogue(const TileArgs& a, TileSmem& s, uint32_t acc_col, int warp, int lane,
                                         int64_t row, int col_tile, int half, int part, RowAhead& ahead, uint64_t* tempty) {
  const bool valid = row < a.rows;
  const int c0 = col_tile + half * 128;
  auto release = [&]() {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_relaxed(mapa_shared(smem_u32(tempty), 0));
  };
  if constexpr (EPI == kStats || EPI == kLogits) {
    if (c0 >= a.cols) {
      release();
      return;
    }
    const int split = c0 / kHeadSplit;
    EntryWalk& en = ahead.en;
    float top = -INFINITY, m = -INFINITY, z = 0.f, u = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float r[32];
      tmem_ld32(acc_col + c * 32, r);
      if (c == 3) release();
      const int col = c0 + c * 32;
      if (col >= a.cols) continue;
      if constexpr (EPI == kStats) {
        if (__any_sync(0xffffffffu, en.cur.x < col + 32)) {
          // a register array cannot be indexed: each lane reads its row back
          stage_row(s.stage[warp - 2], lane, r);
          while (en.cur.x < col + 32) {
            a.picked[row * a.Ntot + en.cur.y] = *staged_at(s.stage[warp - 2], lane, en.cur.x - col);
            en.next();
          }
          __syncwarp();
        }
      }
      mask_columns(r, a.cols - col);
      // four running maxima and sums: the warp's own latency, not the issue rate, is what bounds this epilogue
      float c4[4] = {r[0], r[1], r[2], r[3]};
#pragma unroll
      for (int k = 4; k < 32; ++k) c4[k & 3] = fmaxf(c4[k & 3], r[k]);
      const float cm = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
      if (fabsf(cm) > kLarge) {
        // few instructions (they lie among the others'): from this lane's staged row
        stage_row(s.stage[warp - 2], lane, r);
        const float low = fmaxf(cm, kLowest);
        float lz = 0.f, lu = 0.f;
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
          const float d = low_base2(*staged_at(s.stage[warp - 2], lane, k), a.log2e, low);
          const float e = ex2(d);
          lz += e;
          lu = fmaf(d, e, lu);
        }
        merge_part(m, z, u, low * a.log2e, lz, lu);
        top = fmaxf(top, cm);
      } else {
        if (cm > top) {
          // move the sums to the new reference: with d = m - m', a' = a + d, 2^a' = 2^d 2^a
          const float next = cm * a.log2e;
          if (z > 0.f) {
            const float d = m - next, f = ex2(d);
            u = f > 0.f ? f * fmaf(d, z, u) : 0.f;
            z *= f;
          }
          top = cm;
          m = next;
        }
        float z4[4] = {0.f, 0.f, 0.f, 0.f}, u4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float d = max_nan(to_base2(r[k], a.log2e, m), -200.f);
          const float e = ex2(d);
          z4[k & 3] += e;
          u4[k & 3] = fmaf(d, e, u4[k & 3]);
        }
        z += (z4[0] + z4[1]) + (z4[2] + z4[3]);
        u += (u4[0] + u4[1]) + (u4[2] + u4[3]);
      }
      if constexpr (EPI == kLogits) {
        // through the staging rows: a store instruction writes 4 rows x 128 contiguous bytes
        uint8_t* stage = s.stage[warp - 2];
        stage_row(stage, lane, r);
        __syncwarp();
        const int64_t row0 = row - lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3), ch = lane & 7;
          if (row0 + rr < a.rows)
            *reinterpret_cast<float4*>(a.logits + (row0 + rr) * a.ld + col + ch * 4) = *staged(stage, rr, ch);
        }
        __syncwarp();
      }
    }
    if (valid) a.part[row * a.n_splits + split] = make_float4(m, z, u, top);
  } else if constexpr (EPI == kGrad) {
    if (c0 >= a.gcols) {
      release();
      return;
    }
    const float4 ri = ahead.ri;
    const bool live = valid && !(ri.w == 0.f);
    const bool all_live = __all_sync(0xffffffffu, live);
    const float lse2 = ri.x * kLog2e, A = ri.y, B2 = ri.z * kLn2;
    EntryWalk& en = ahead.en;
    uint8_t* stage = s.stage[warp - 2];
    const int64_t piece_row = row - lane + (lane >> 2);
    const int64_t left_rows = a.rows - piece_row;
    uint8_t* dst = reinterpret_cast<uint8_t*>(a.G + piece_row * a.ld + c0 + (lane & 3) * 8);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float r[32];
      tmem_ld32(acc_col + c * 32, r);
      if (c == 3) release();
      const int col = c0 + c * 32;
      if (col >= a.gcols) continue;
      const int left = a.cols - col;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float d = to_base2(r[k], a.log2e, lse2);
        r[k] = ex2(d) * fmaf(B2, max_nan(d, -200.f), A);           // 2^-200 is 0 to ex2; d may be as low as a mask
      }
      if (!all_live || left < 32) {
#pragma unroll
        for (int k = 0; k < 32; ++k) r[k] = live && k < left ? r[k] : 0.f;
      }
      if (__any_sync(0xffffffffu, en.cur.x - a.v0 < col + 32)) {
        stage_row(stage, lane, r);
        while (en.cur.x - a.v0 < col + 32) {
          *staged_at(stage, lane, en.cur.x - a.v0 - col) += __int_as_float(en.cur.y);
          en.next();
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 v = *staged(stage, lane, k);
          r[4 * k] = v.x;
          r[4 * k + 1] = v.y;
          r[4 * k + 2] = v.z;
          r[4 * k + 3] = v.w;
        }
        __syncwarp();                      // the rows below lie across these
      }
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = pack_g2(r[2 * k], r[2 * k + 1]);
      store_pairs(stage, lane, w, dst + c * 64, a.ld * 2, left_rows);
    }
  } else {
    // the operands' scales taken out: of the copy of h, or of the copy of W and the row of G'
    float f1, f2 = 1.f;
    if constexpr (EPI == kDw) f1 = __uint_as_float(*a.smax) / kRowLift;
    else split_scale(*a.inv, valid ? a.row[row].w : 0.f, f1, f2);
    const auto scaled = [&](float v) { return EPI == kDw ? v * f1 : v * f1 * f2; };
    uint8_t* stage = s.stage[warp - 2];
    const int64_t row0 = row - lane;
    if (OUT_BF16 && (EPI == kDw || a.acc == nullptr)) {
      const int64_t piece_row = row0 + (lane >> 2);
      uint8_t* dst = reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(a.out) + piece_row * a.cols + c0 + (lane & 3) * 8);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float r[32];
        tmem_ld32(acc_col + c * 32, r);
        if (c == 3) release();
        if (c0 + c * 32 >= a.cols) continue;
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = pack_bf16x2(scaled(r[2 * k]), scaled(r[2 * k + 1]));
        store_pairs(stage, lane, w, dst + c * 64, static_cast<int64_t>(a.cols) * 2, a.rows - piece_row);
      }
    } else if constexpr (!(OUT_BF16 && EPI == kDw)) {
      // fp32 out, or earlier chunks' sums to add before the rounding: fp32 through the staging rows
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float r[32];
        tmem_ld32(acc_col + c * 32, r);
        if (c == 3) release();
        const int col = c0 + c * 32;
        if (col >= a.cols) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) r[k] = scaled(r[k]);
        stage_row(stage, lane, r);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3), ch = lane & 7;
          if (row0 + rr >= a.rows) continue;
          float4 v = *staged(stage, rr, ch);
          const int64_t off = (row0 + rr) * a.cols + col + ch * 4;
          if constexpr (OUT_BF16) {
            const float4 o = *reinterpret_cast<const float4*>(a.acc + off);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + off) =
                make_uint2(pack_bf16x2(v.x + o.x, v.y + o.y), pack_bf16x2(v.z + o.z, v.w + o.w));
          } else {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) +
                                                    static_cast<int64_t>(part) * a.rows * a.cols + off);
            if (a.accumulate) {
              const float4 o = *dst;
              v.x += o.x;
              v.y += o.y;
              v.z += o.z;
              v.w += o.w;
            }
            *dst = v;
          }
        }
        __syncwarp();
      }
    }
  }
}

template <Epi EPI>
constexpr int threads_of() { return EPI == kGrad ? kThreads + kCopyThreads : kThreads; }

template <Epi EPI, bool OUT_BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of<EPI>(), 1)
    head_tile_kernel(const __grid_constant__ TileMaps maps, const TileArgs a) {
  using L = Layout<EPI>;
  extern __shared__ uint8_t smem_raw[];
  TileSmem& s = *reinterpret_cast<TileSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &s.abort;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], 2 * kEpiWarps);
    }
    mbar_init(&s.drain, 1);
    s.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s.tmem_base, 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();        // every barrier of both CTAs exists before any remote arrive
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  after_previous();

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int i = pair; i < a.units && ok; i += npairs) {
        const Unit u = unit_at(a, i);
        const int row0 = u.mt * 2 * kBM + static_cast<int>(rank) * kBM;    // this CTA's rows of A
        const int n0 = u.nt * kBN + static_cast<int>(rank) * (kBN / 2);    // and of B
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!mbar_wait(&s.empty[stage], phase ^ 1, abort, a.status)) { ok = false; break; }
          const uint32_t lfull = mapa_shared(smem_u32(&s.full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(&s.full[stage], 2 * (kBM + kBN / 2) * kBK * 2);
          if (L::a_mn) {
#pragma unroll
            for (int j = 0; j < kBM / 64; ++j)
              tma_load_2d_pair(&maps.a, lfull, s.a[stage] + j * (64 * kBK * 2), row0 + j * 64, kb * kBK);
          } else {
            tma_load_2d_pair(&maps.a, lfull, s.a[stage], kb * kBK, row0);
          }
          if (L::b_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d_pair(&maps.b, lfull, s.b[stage] + j * (64 * kBK * 2), n0 + j * 64, kb * kBK);
          } else {
            tma_load_2d_pair(&maps.b, lfull, s.b[stage], kb * kBK, n0);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        // this CTA's loads complete on the leader's barrier: give them time to land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (leader CTA)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = L::f16 ? idesc_f16(2 * kBM, kBN, L::a_mn, L::b_mn)
                                        : idesc_bf16(2 * kBM, kBN, L::a_mn, L::b_mn);
      // one tcgen05.mma further along K: 32 bytes inside the swizzled row, or 16 rows of 128 bytes
      constexpr uint32_t a_step = L::a_mn ? (kUK * 128) >> 4 : (kUK * 2) >> 4;
      constexpr uint32_t b_step = L::b_mn ? (kUK * 128) >> 4 : (kUK * 2) >> 4;
      constexpr uint32_t a_lbo = L::a_mn ? 64 * kBK * 2 : 16;
      constexpr uint32_t b_lbo = L::b_mn ? 64 * kBK * 2 : 16;
      uint32_t stage = 0, phase = 0, iter = 0;
      bool ok = true;
      for (int i = pair; i < a.units && ok; i += npairs, ++iter) {
        const Unit u = unit_at(a, i);
        const uint32_t buf = iter & 1;
        if (!mbar_wait(&s.tempty[buf], ((iter >> 1) & 1) ^ 1, abort, a.status)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * kBN;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!mbar_wait(&s.full[stage], phase, abort, a.status)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(smem_u32(s.a[stage]), a_lbo, 1024);
          const uint64_t db = smem_desc_sw128(smem_u32(s.b[stage]), b_lbo, 1024);
#pragma unroll
          for (int k = 0; k < kBK / kUK; ++k)
            umma_bf16_pair(d, da + static_cast<uint64_t>(k * a_step), db + static_cast<uint64_t>(k * b_step), idesc,
                           kb > u.kb0 || k > 0);
          const uint32_t e = smem_u32(&s.empty[stage]);
          umma_commit_pair(mapa_shared(e, 0));
          umma_commit_pair(mapa_shared(e, 1));
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (ok) {
          const uint32_t f = smem_u32(&s.tfull[buf]);
          umma_commit_pair(mapa_shared(f, 0));
          umma_commit_pair(mapa_shared(f, 1));
        }
      }
      umma_commit_pair(mapa_shared(smem_u32(&s.drain), 0));
      int dummy = 0;
      (void)mbar_wait(&s.drain, 0, &dummy, a.status);     // every MMA done before TMEM is released
    }
  } else if (warp < 2 + kEpiWarps) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;                               // TMEM lane quadrant this warp may read
    const int half = (warp - 2) >> 2;
    const uint32_t base = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
    uint32_t iter = 0;
    for (int i = pair; i < a.units; i += npairs, ++iter) {
      const Unit u = unit_at(a, i);
      const uint32_t buf = iter & 1;
      const int64_t row = static_cast<int64_t>(u.mt) * 2 * kBM + rank * kBM + q * 32 + lane;
      RowAhead ahead;
      if constexpr (EPI == kStats || EPI == kGrad) {
        const int c0 = u.nt * kBN + half * 128;
        if constexpr (EPI == kGrad) ahead.ri = row < a.rows ? a.row[row] : make_float4(0.f, 0.f, 0.f, 0.f);
        // (a row of scale 0 has entries, of coefficient 0: its G' is 0 whatever the row holds)
        ahead.en.start(a, row < a.rows && c0 < a.cols, static_cast<int>(row), (a.v0 + c0) / kHeadSplit);
      }
      if (!warp_wait(&s.tfull[buf], (iter >> 1) & 1, abort, a.status)) break;
      tc_fence_after();
      epilogue<EPI, OUT_BF16>(a, s, base + buf * kBN, warp, lane, row, u.nt * kBN, half, u.part, ahead,
                              &s.tempty[buf]);
    }
  } else if constexpr (EPI == kGrad) {
    // ---------------------------------------------------------------- fp16 copies for dh and dw
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x - kThreads;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kCopyThreads;
    if (a.w_copied) rescale_w(a.copy_w, first, stride);
    else if (a.copy_w.n_vec > 0) copy_w(a.copy_w, first, stride);
    copy_h(a.copy_h, first, stride);
  }

  __syncthreads();
  tc_fence_before();
  cluster_sync_all();        // no CTA leaves while its pair may still touch its memory
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

// dh from the parts of a split K, summed in order: into acc, or with acc (may
// be NULL) to bf16.
struct ReduceArgs {
  const float4* part;              // [parts][n] of four values
  int parts;
  int64_t n;
  float4* acc;
  int acc_in;                      // acc holds earlier chunks
  uint2* out;                      // bf16, or NULL: the sums go to acc
};

// Eight lanes per output, each with every eighth part; their sums meet in a
// fixed order.
constexpr int kReduceLanes = 8;

__global__ void __launch_bounds__(256) head_reduce_kernel(const ReduceArgs a) {
  after_previous();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kReduceLanes;
  const int own = threadIdx.x % kReduceLanes;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < a.n) {
    if (own == 0 && a.acc_in) v = a.acc[i];
#pragma unroll 4
    for (int p = own; p < a.parts; p += kReduceLanes) {
      const float4 x = a.part[p * a.n + i];
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
  }
#pragma unroll
  for (int o = kReduceLanes / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
  }
  if (i >= a.n || own != 0) return;
  if (a.out == nullptr) {
    a.acc[i] = v;
    return;
  }
  a.out[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

constexpr int kMaxDevices = 64;

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) (void)cudaGetLastError();
  return dev;
}

}  // namespace

bool head_make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int box_inner,
                   int box_outer, bool fp16) {
  EncodeTiledFn enc = get_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int head_num_sms() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = current_device();
  int n = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n = 148;
    if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

namespace {

constexpr size_t kSmemBytes = sizeof(TileSmem) + 1024;

// CTA pairs that can be resident at once: a persistent grid larger than that
// would leave whole pairs waiting for a second wave.  Asked once per kernel and
// device (a property of both): the query costs the host more than a launch.
template <Epi EPI, bool OUT_BF16>
int resident_pairs() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = current_device();
  if (dev < kMaxDevices && known[dev].load(std::memory_order_relaxed) > 0)
    return known[dev].load(std::memory_order_relaxed);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(head_num_sms()));
  cfg.blockDim = dim3(threads_of<EPI>());
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, head_tile_kernel<EPI, OUT_BF16>, &cfg) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    return head_num_sms() / 2;
  }
  if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

int tiles_of(int64_t extent, int64_t tile) { return static_cast<int>((extent + tile - 1) / tile); }

// parts: how many parts K is cut into (dh).
template <Epi EPI, bool OUT_BF16>
cudaError_t run_tiles(const TileMaps& maps, TileArgs a, int64_t kdim, int parts, cudaStream_t st) {
  a.n_mt = tiles_of(a.rows, 2 * kBM);
  a.n_nt = tiles_of(EPI == kGrad ? a.gcols : a.cols, kBN);
  a.kblocks = tiles_of(kdim, kBK);
  a.part_kblocks = tiles_of(a.kblocks, parts);
  a.parts = tiles_of(a.kblocks, a.part_kblocks);
  const int64_t units = static_cast<int64_t>(a.n_mt) * a.n_nt * a.parts;
  if (units > INT32_MAX - 1024) return cudaErrorInvalidValue;
  a.units = static_cast<int>(units);
  auto fn = head_tile_kernel<EPI, OUT_BF16>;
  cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (err != cudaSuccess) return err;
  const int resident = resident_pairs<EPI, OUT_BF16>();
  const int pairs = a.units < resident ? a.units : resident;
  return head_launch(fn, dim3(static_cast<unsigned>(2 * pairs)), threads_of<EPI>(), kSmemBytes, st, maps, a);
}

// Parts of dh's K: dh has ceil(T / 256) ceil(D / 256) tiles, few when T is
// small, and K = V is long.  The count with the least of (turns of the pairs x
// K per turn at 0.3 us per 64) + (the parts' fp32 sums, written and read, at
// 5 TB/s, and one more launch), if that is under 0.8 of one part's: with 1.7
// tiles per pair (T = 8192, D = 1024) parts measured 608 us and one part 573 to
// 618, the power cap and not the turns setting the time.
int dh_parts(int64_t T, int64_t D, int64_t V) {
  constexpr int kPairs = 74;
  const double tiles = static_cast<double>(tiles_of(T, 2 * kBM)) * tiles_of(D, kBN);
  const int kb = tiles_of(V, kBK);
  int best = 1;
  double least = 0.0, one = 0.0;
  for (int p = 1; p <= kPairs && p <= kb; ++p) {
    const double turns = static_cast<double>(static_cast<int64_t>((tiles * p + kPairs - 1) / kPairs));
    double us = turns * tiles_of(kb, p) * 0.3;
    if (p > 1) us += static_cast<double>(p) * T * D * 8.0 / 5.0e6 + 3.0;
    if (p == 1) one = least = us;
    if (us < least && us < 0.8 * one) {
      best = p;
      least = us;
    }
  }
  return best;
}

// Backward workspace: [G' chunk: T x round_up(Vc, 64) f16][dh partial sums:
// T x D f32, only with more than one chunk][parts of dh: T x D f32 each][h in
// fp16][the chunk's W rows in fp16][copy scales].
struct BwdWs {
  int64_t ldg;
  int parts;
  size_t g, acc, part, h16, w16, aux;
  size_t total() const { return g + acc + part + h16 + w16 + aux; }
};

BwdWs bwd_layout(const HeadProblem& p, int64_t Vc) {
  BwdWs w{};
  w.ldg = (Vc + 63) / 64 * 64;
  w.g = head_align(static_cast<size_t>(p.T) * w.ldg * 2);
  w.acc = Vc < p.V ? head_align(static_cast<size_t>(p.T) * p.D * 4) : 0;
  w.parts = dh_parts(p.T, p.D, p.V);
  w.part = w.parts > 1 ? head_align(static_cast<size_t>(w.parts) * p.T * p.D * 4) : 0;
  w.h16 = head_align(static_cast<size_t>(p.T) * p.D * 2);
  w.w16 = head_align(static_cast<size_t>(Vc) * p.D * 2);
  w.aux = 256;                       // W's copy scale
  return w;
}

}  // namespace

cudaError_t head_tc_forward(const HeadProblem& p, const HeadForward& f, cudaStream_t st) {
  TileMaps maps;
  if (!head_make_map(&maps.a, f.h, p.D, f.T, p.D, kBK, kBM, false)) return cudaErrorInvalidValue;
  if (!head_make_map(&maps.b, p.W, p.D, p.V, p.D, kBK, kBN / 2, false)) return cudaErrorInvalidValue;
  TileArgs a{};
  a.rows = static_cast<int>(f.T);
  a.cols = static_cast<int>(p.V);
  a.n_splits = static_cast<int>(head_splits(p.V));
  a.part = f.part;
  a.log2e = head_log2e(p.D, 1);
  a.logits = f.logits;
  a.ld = f.ld;
  a.e = f.en.e;
  a.first = f.en.first;
  a.ld_first = f.ld_first;
  a.Ntot = f.en.Ntot;
  a.picked = f.picked;
  a.status = p.status;
  return f.logits != nullptr ? run_tiles<kLogits, false>(maps, a, p.D, 1, st)
                             : run_tiles<kStats, false>(maps, a, p.D, 1, st);
}

size_t head_tc_bwd_bytes(const HeadProblem& p, int64_t Vc) { return bwd_layout(p, Vc).total(); }

// The widest chunk (the whole vocabulary, or equal chunks of a multiple of 256
// columns) whose workspace fits; 0 when none does.
int64_t head_tc_bwd_chunk(const HeadProblem& p, size_t budget) {
  if (bwd_layout(p, p.V).total() <= budget) return p.V;
  int64_t lo = 0, hi = (p.V - 1) / kBN;                 // chunks of kBN columns
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (bwd_layout(p, mid * kBN).total() <= budget) lo = mid; else hi = mid - 1;
  }
  if (lo == 0) return 0;
  const int64_t n = (p.V + lo * kBN - 1) / (lo * kBN);
  const int64_t even = ((p.V + n - 1) / n + kBN - 1) / kBN * kBN;
  return even < lo * kBN ? even : lo * kBN;
}

cudaError_t head_tc_backward(const HeadProblem& p, const HeadEntriesIn& in, const HeadEntries& en, void* dh, void* dW,
                             bool dW_bf16, int accumulate, void* ws, int64_t Vc, cudaStream_t st) {
  const BwdWs w = bwd_layout(p, Vc);
  char* q = static_cast<char*>(ws);
  __half* G = reinterpret_cast<__half*>(q);
  q += w.g;
  float* acc = w.acc != 0 ? reinterpret_cast<float*>(q) : nullptr;
  q += w.acc;
  float* part = reinterpret_cast<float*>(q);
  q += w.part;
  __half* h16 = reinterpret_cast<__half*>(q);
  q += w.h16;
  __half* w16 = reinterpret_cast<__half*>(q);
  q += w.w16;
  float* inv = reinterpret_cast<float*>(q);
  cudaError_t err = cudaSuccess;
  // From 512 tokens on the tensor pipe bounds the G' kernel and two more warps of it copy W beside it; below, reading W
  // bounds it and the copy, in so few threads, would prolong it: further blocks of the entries' launch make it.  Whole
  // steps, V = 32771, D = 1024, beside and before: T = 300 215 and 201 us, 777 265 and 278, 1200 329 and 354, 2047 530
  // and 535.
  const bool beside = p.T >= 512;
  for (int64_t v0 = 0; v0 < p.V; v0 += Vc) {
    const int64_t n = v0 + Vc <= p.V ? Vc : p.V - v0;
    const bool first = v0 == 0, last = v0 + n >= p.V;
    const void* Wc = static_cast<const __nv_bfloat16*>(p.W) + v0 * p.D;
    HeadCopyW w_copy{};
    if (dh != nullptr) w_copy = HeadCopyW{Wc, w16, n * p.D / 8, en.smax + 1, inv};
    if (first) {
      err = run_head_entries(in, en, true, p.status, beside || dh == nullptr ? nullptr : &w_copy, st);
      if (err != cudaSuccess) return err;
    } else if (dh != nullptr) {
      err = cudaMemsetAsync(en.smax + 1, 0, sizeof(unsigned int), st);
      if (err != cudaSuccess) return err;
      if (!beside) {
        err = head_launch(head_copy_kernel, dim3(head_copy_blocks(w_copy.n_vec)), 256, 0, st, w_copy);
        if (err != cudaSuccess) return err;
      }
    }
    TileMaps maps;
    TileArgs a{};
    a.status = p.status;
    // G' of the chunk
    if (!head_make_map(&maps.a, p.h, p.D, p.T, p.D, kBK, kBM, false)) return cudaErrorInvalidValue;
    if (!head_make_map(&maps.b, Wc, p.D, n, p.D, kBK, kBN / 2, false)) return cudaErrorInvalidValue;
    a.rows = static_cast<int>(p.T);
    a.cols = static_cast<int>(n);
    a.v0 = static_cast<int>(v0);
    a.log2e = head_log2e(p.D, 1);
    a.e = en.e;
    a.first = en.first;
    a.ld_first = p.T;
    a.Ntot = en.Ntot;
    a.row = en.row;
    a.G = G;
    a.ld = w.ldg;
    a.gcols = static_cast<int>((n + 63) / 64 * 64);
    a.copy_w = w_copy;
    a.w_copied = beside ? 0 : 1;
    if (dW != nullptr && first)
      a.copy_h = HeadCopyH{p.h, h16, p.T * p.D / 8, static_cast<int>(p.D / 8), en.row, en.smax};
    err = run_tiles<kGrad, false>(maps, a, p.D, 1, st);
    if (err != cudaSuccess) return err;
    const HeadExact exact{p.T, p.D, p.h, p.W, en, G, w.ldg, v0, n};
    err = run_head_exact(exact, dh != nullptr && beside ? &w_copy : nullptr, st);
    if (err != cudaSuccess) return err;
    if (dh != nullptr) {
      TileArgs d{};
      d.status = p.status;
      d.rows = static_cast<int>(p.T);
      d.cols = static_cast<int>(p.D);
      d.inv = inv;
      d.row = en.row;
      if (!head_make_map(&maps.a, G, a.gcols, p.T, w.ldg, kBK, kBM, true)) return cudaErrorInvalidValue;
      if (!head_make_map(&maps.b, w16, p.D, n, p.D, 64, kBK, true)) return cudaErrorInvalidValue;
      if (w.parts > 1) {
        d.out = part;
        err = run_tiles<kDh, false>(maps, d, n, w.parts, st);
        if (err != cudaSuccess) return err;
        ReduceArgs r{};
        r.part = reinterpret_cast<const float4*>(part);
        const int kb = tiles_of(n, kBK);
        r.parts = tiles_of(kb, tiles_of(kb, w.parts));
        r.n = p.T * p.D / 4;
        r.acc = reinterpret_cast<float4*>(acc);
        r.acc_in = first ? 0 : 1;
        r.out = last ? static_cast<uint2*>(dh) : nullptr;
        err = head_launch(head_reduce_kernel, dim3(static_cast<unsigned>((r.n * kReduceLanes + 255) / 256)), 256, 0, st,
                          r);
      } else if (last) {
        d.out = dh;
        d.acc = first ? nullptr : acc;
        err = run_tiles<kDh, true>(maps, d, n, 1, st);
      } else {
        d.out = acc;
        d.accumulate = first ? 0 : 1;
        err = run_tiles<kDh, false>(maps, d, n, 1, st);
      }
      if (err != cudaSuccess) return err;
    }
    if (dW != nullptr) {
      TileArgs d{};
      d.status = p.status;
      d.rows = static_cast<int>(n);
      d.cols = static_cast<int>(p.D);
      d.smax = en.smax;
      d.accumulate = accumulate;
      if (!head_make_map(&maps.a, G, a.gcols, p.T, w.ldg, 64, kBK, true)) return cudaErrorInvalidValue;
      if (!head_make_map(&maps.b, h16, p.D, p.T, p.D, 64, kBK, true)) return cudaErrorInvalidValue;
      if (dW_bf16) {
        d.out = static_cast<__nv_bfloat16*>(dW) + v0 * p.D;
        err = run_tiles<kDw, true>(maps, d, p.T, 1, st);
      } else {
        d.out = static_cast<float*>(dW) + v0 * p.D;
        err = run_tiles<kDw, false>(maps, d, p.T, 1, st);
      }
      if (err != cudaSuccess) return err;
    }
  }
  return cudaSuccess;
}

}  // namespace mls
