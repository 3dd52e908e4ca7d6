// Host helpers shared by the tensor-core files of the single-exit operators.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <utility>

#include "kernels.h"

namespace mls {

// 2-D tensor of 16-bit elements [outer][ld], the first `inner` of each row
// addressable (elements outside read as zero), 128-byte swizzled boxes.  False
// when the driver's encoder is missing or refuses.
bool head_make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int box_inner,
                   int box_outer, bool fp16);

// SMs of the current device.
int head_num_sms();

// Blocks of 256 threads for a copy of n_vec vectors.
inline unsigned head_copy_blocks(int64_t n_vec) {
  const int64_t want = (n_vec + 2047) / 2048, cap = 8 * static_cast<int64_t>(head_num_sms());
  return static_cast<unsigned>(want < 1 ? 1 : want < cap ? want : cap);
}

// Launches a kernel that calls after_previous() (head_dev.cuh) before it touches
// global memory: it may be set up while the one before it on the stream ends.
// A step of a few tokens is ten launches of a few microseconds each, of which
// the gaps were a sixth.
template <typename... P, typename... A>
cudaError_t head_launch(void (*fn)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, fn, std::forward<A>(args)...);
  note_launches(1);
  return err;
}

}  // namespace mls
