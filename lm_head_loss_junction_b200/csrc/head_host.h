// Host helpers shared by the tensor-core files of the single-exit operators.
#pragma once
#include <cuda.h>
#include <cstdint>

namespace mls {

// 2-D tensor of 16-bit elements [outer][ld], the first `inner` of each row
// addressable (elements outside read as zero), 128-byte swizzled boxes.  False
// when the driver's encoder is missing or refuses.
bool head_make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int box_inner,
                   int box_outer, bool fp16);

// SMs of the current device.
int head_num_sms();

}  // namespace mls
