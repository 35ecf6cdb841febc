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
constexpr int kStreamSmem = 226 << 10;  // shared memory per SM the streaming form plans with
constexpr int kStreamStatic = 2048;     // of which a CTA's static part and the runtime's reserve
constexpr int kStreamStages = 8;        // stages per CTA at most
constexpr int kStreamCtas = 16;         // CTAs per SM at most
cudaError_t launch_combine_norm(const void* y, bool y_f32, bool pair_order,
                                const int32_t* row_of_pair, int T, int k, int H, const TailP& p,
                                int* status, int sms, cudaStream_t st);

}  // namespace moe
