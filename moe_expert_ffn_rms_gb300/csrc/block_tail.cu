// moe_combine_norm: the sum of a token's expert rows and what follows the
// block (block_tail.cuh) in one pass over the data.
#include "block_tail.cuh"
#include "kernels.h"
#include "tail.h"

namespace moe {
namespace {

// One CTA per token; thread `tid` holds the 8-column chunks tid, tid +
// blockDim, ... (at most VPT) in registers from the first read to the last
// write, so each input is read once and each output written once.
template <int VPT>
__global__ void __launch_bounds__(1024) combine_norm_kernel(
    const void* __restrict__ y, int y_f32, int pair_order, const int32_t* __restrict__ row_of_pair,
    int T, int k, int H, const TailP p, int* status) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[32];
  const int t = blockIdx.x;
  const int nv = H >> 3;
  float f[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
  for (int j = 0; j < k; ++j) {  // summed in slot order, skipped pairs excluded
    const int64_t pair = (int64_t)t * k + j;
    int64_t row = pair;
    if (row_of_pair) {
      const int r = row_of_pair[pair];
      if (r < 0) continue;
      if (r >= T * k) {
        if (threadIdx.x == 0) flag_status(status, MOE_ERR_INVALID_ARG);
        continue;
      }
      if (!pair_order) row = r;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= nv) break;
      float a[8];
      load8(y, y_f32 != 0, (size_t)row * H + v * 8, a);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[i][q] += a[q];
    }
  }
  float r = 1.f;
  if (p.post_w) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(f[i][q], f[i][q], ss);
    r = 1.0f / sqrtf(block_sum(ss, red) / (float)H + p.post_eps);
  }
  const int grow = tail_gate_row(p, t, threadIdx.x == 0 ? status : nullptr);
  const float factor = tail_row_factor(p, grow);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v >= nv) break;
    float h[8];
    tail_h8(p, t, H, v * 8, f[i], r, grow, factor, h);
    store8(p.out, p.out_f32 != 0, (size_t)t * H + v * 8, h);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      f[i][q] = h[q];
      ss = fmaf(h[q], h[q], ss);
    }
  }
  if (!p.next_w) return;
  r = 1.0f / sqrtf(block_sum(ss, red) / (float)H + p.next_eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    float m = 0.f;
    if (v < nv) {
      float w[8];
      load8(p.next_w, false, v * 8, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[i][q] = (f[i][q] * r) * w[q];
        m = fmaxf(m, fabsf(f[i][q]));
      }
      if (p.xhat) store8_bf16(p.xhat + (size_t)t * H + v * 8, f[i]);
    }
    if (p.xq && p.q_group) {
      // a group of 128 columns is 16 consecutive lanes (blockDim is a
      // multiple of 32, H of 128)
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = m > 0.f ? __fdiv_rn(m, 448.0f) : 1.0f;
      if (v < nv) {
        *reinterpret_cast<uint2*>(p.xq + (size_t)t * H + v * 8) = tail_e4m3x8(f[i], s);
        if ((v & 15) == 0) p.xscale[(size_t)t * (H >> 7) + (v >> 4)] = s;
      }
    }
    amax = fmaxf(amax, m);
  }
  if (p.xq && !p.q_group) {
    amax = block_max(amax, red);
    const float s = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nv) *reinterpret_cast<uint2*>(p.xq + (size_t)t * H + v * 8) = tail_e4m3x8(f[i], s);
    }
    if (threadIdx.x == 0) p.xscale[t] = s;
  }
}

}  // namespace

cudaError_t launch_combine_norm(const void* y, bool y_f32, bool pair_order,
                                const int32_t* row_of_pair, int T, int k, int H, const TailP& p,
                                int* status, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const int nv = H / 8;
  int threads = rmsnorm_threads(T, nv);
  if (threads * 4 < nv) threads = ((nv + 3) / 4 + 31) / 32 * 32;
  const int vpt = (nv + threads - 1) / threads;
#define MOE_CN(V)                                                                              \
  return launch_kernel(combine_norm_kernel<V>, dim3(T), dim3(threads), 0, st, y, (int)y_f32,   \
                       (int)pair_order, row_of_pair, T, k, H, p, status)
  if (vpt <= 1) MOE_CN(1);
  if (vpt <= 2) MOE_CN(2);
  MOE_CN(4);
#undef MOE_CN
}

}  // namespace moe
