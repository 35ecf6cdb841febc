// Sums over the rows of partial results, used by the gradients that reduce over a batch.
#pragma once

#include "common.cuh"

namespace moe {

// out0[c] (c < split) / out1[c - split] = sum over i < n of part[i * pitch + c], c < cols, in a
// fixed order: COLS columns per CTA, 1024 / COLS threads on each.
template <int COLS>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ part, int n, int64_t pitch,
                                                          int64_t cols, int64_t split, float* out0, float* out1) {
  constexpr int Y = 1024 / COLS;
  __shared__ float red[Y][COLS + 1];
  pdl_trigger();
  pdl_wait();
  const int x = threadIdx.x % COLS, y = threadIdx.x / COLS;
  const int64_t c = (int64_t)blockIdx.x * COLS + x;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int i = y; i < n; i += Y) s += part[i * pitch + c];
  }
  red[y][x] = s;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int w = threadIdx.x >> 5; w < COLS; w += 32) {
    s = 0.f;
    for (int i = lane; i < Y; i += 32) s += red[i][w];
    s = warp_sum(s);
    const int64_t o = (int64_t)blockIdx.x * COLS + w;
    if (lane != 0 || o >= cols) continue;
    if (o < split) out0[o] = s;
    else out1[o - split] = s;
  }
}

// Few columns per CTA (many threads on each) as long as all CTAs run at once: 608 rows of
// 4096 columns 9.6 us with 8 threads per column and 128 CTAs, below 3 with 64.  By the
// pitch, so that a call that leaves out the second output adds the first in the same order.
inline cudaError_t launch_column_sum(const float* part, int n, int64_t pitch, int64_t cols, int64_t split, float* out0,
                                     float* out1, int sms, cudaStream_t st) {
  auto kern = column_sum_kernel<16>;
  int per = 16;
  if (pitch > (int64_t)per * 2 * sms) {
    kern = column_sum_kernel<32>;
    per = 32;
  }
  if (pitch > (int64_t)per * 2 * sms) {
    kern = column_sum_kernel<64>;
    per = 64;
  }
  return launch_kernel(kern, dim3((unsigned)((cols + per - 1) / per)), dim3(1024), 0, st, part, n, pitch, cols, split,
                       out0, out1);
}

}  // namespace moe
