// Host-side launch functions of the fused block tail and the few-token layer
// (internal to libmoeffn).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "block_tail.cuh"

namespace moe {

// moe_combine_norm; H <= kTailMaxH.
constexpr int kTailMaxH = 32768;
cudaError_t launch_combine_norm(const void* y, bool y_f32, bool pair_order,
                                const int32_t* row_of_pair, int T, int k, int H, const TailP& p,
                                int* status, cudaStream_t st);

}  // namespace moe
