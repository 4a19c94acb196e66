// evict.h -- launcher of the eviction kernels (evict.cu).  Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"
#include "sa.h"

namespace sa {

// Workspace of sa_evict_tokens: status | src_row int32 [batch, budget] |
// kept int32 [batch] | fault int32 [batch].
inline size_t evict_kept_offset(int32_t batch, int32_t budget) {
    return kStatusBytes + (size_t)round_up((int64_t)batch * budget * 4, 256);
}

cudaError_t launch_evict(const sa_cache *src, const float *acc, int64_t ld_acc, int32_t budget,
                         int32_t keep_first, int32_t keep_last, const sa_cache *dst,
                         float *acc_out, int64_t ld_out, int32_t *src_pos, void *workspace,
                         cudaStream_t s);

}  // namespace sa
