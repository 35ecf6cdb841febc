// Expert rows back to their tokens with the routing weights applied
// (moe_unpermute), the gradients of that (moe_unpermute_backward) and of the
// gather that sorted the tokens by expert (moe_permute_backward, the same sum
// without weights).
//
//   out[t]   = residual[t] + sum_j w[t,j] y[r(t,j)]
//   dy[r(t,j)] = w[t,j] dout[t],   dw[t,j] = <dout[t], y[r(t,j)]>
//   dlogits[t,e] = sum_{j: ids[t,j] = e} w_j (dw_j - sum_i w_i dw_i)
//
// Every row is read once and every result written once, so the bound is the
// copy bandwidth.
#include "block_tail.cuh"
#include "common.cuh"
#include "train.h"

namespace moe {
namespace {

// Row of pair (t, j), or -1 when the pair has none.
MOE_DEV int pair_row(const int32_t* row_of_pair, int64_t pair, int rows, bool flag, int* status) {
  const int r = row_of_pair[pair];
  if (r < rows) return r;
  if (flag) flag_status(status, MOE_ERR_INVALID_ARG);
  return -1;
}

constexpr int kRowsThreads = 256;

// A thread takes 8 columns of a token: its k rows' loads are all issued before
// the first use.  blockDim = (column chunks, tokens).
template <int KB, bool YF32>
__global__ void __launch_bounds__(kRowsThreads) unpermute_kernel(const UnpermuteArgs a, int* status) {
  pdl_trigger();
  pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int v = blockIdx.y * blockDim.x + threadIdx.x, nv = a.H >> 3;
  if (t >= a.T || v >= nv) return;
  int row[KB];
  float w[KB];
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    row[j] = -1;
    w[j] = 1.f;
    if (j < a.k) {
      row[j] = pair_row(a.row_of_pair, t * a.k + j, a.T * a.k, v == 0, status);
      if (a.w) w[j] = a.w[t * a.k + j];
    }
  }
  constexpr int W = YF32 ? 2 : 1;
  uint4 q[KB][W];
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    if (row[j] >= 0) {
      const uint4* s = static_cast<const uint4*>(a.y) + ((int64_t)row[j] * nv + v) * W;
#pragma unroll
      for (int i = 0; i < W; ++i) q[j][i] = s[i];
    }
  }
  float f[8] = {};
  if (a.residual) load8(a.residual, a.res_f32, (size_t)t * a.H + v * 8, f);
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    if (row[j] < 0) continue;
    float b[8];
    if (YF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = __uint_as_float((&q[j][0].x)[i]);
    } else {
      unpack8_bf16(q[j][0], b);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf(w[j], b[i], f[i]);
  }
  store8(a.out, a.out_f32, (size_t)t * a.H + v * 8, f);
}

// blockDim = (threads of a token, a multiple of 32; tokens).
template <int KB, bool YF32>
__global__ void __launch_bounds__(kRowsThreads) unpermute_grad_kernel(const UnpermuteGradArgs a,
                                                                      int* status) {
  __shared__ float red[kRowsThreads / 32][KB];
  pdl_trigger();
  pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int nv = a.H >> 3, tx = threadIdx.x, nt = blockDim.x;
  const bool on = t < a.T;
  int row[KB];
  float w[KB], dot[KB];
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    row[j] = -1;
    w[j] = dot[j] = 0.f;
    if (on && j < a.k) {
      row[j] = pair_row(a.row_of_pair, t * a.k + j, a.T * a.k, tx == 0, status);
      w[j] = a.w[t * a.k + j];
    }
  }
  const bool dots = a.dw || a.dlogits;
  constexpr int W = YF32 ? 2 : 1;
  for (int v = tx; on && v < nv; v += nt) {
    float d[8];
    uint4 q[KB][W];
    if (dots) {
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (row[j] >= 0) {
          const uint4* s = static_cast<const uint4*>(a.y) + ((int64_t)row[j] * nv + v) * W;
#pragma unroll
          for (int i = 0; i < W; ++i) q[j][i] = s[i];
        }
      }
    }
    load8(a.dout, a.dout_f32, (size_t)t * a.H + v * 8, d);
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      if (row[j] < 0) continue;
      if (dots) {
        float b[8];
        if (YF32) {
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = __uint_as_float((&q[j][0].x)[i]);
        } else {
          unpack8_bf16(q[j][0], b);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], b[i], dot[j]);
      }
      if (a.dy) {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = w[j] * d[i];
        store8(a.dy, YF32, (size_t)row[j] * a.H + v * 8, g);
      }
    }
  }
  if (!dots) return;
  const int warp0 = threadIdx.y * (nt >> 5);
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    dot[j] = warp_sum(dot[j]);
    if ((tx & 31) == 0) red[warp0 + (tx >> 5)][j] = dot[j];
  }
  __syncthreads();
  if (!on) return;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    dot[j] = 0.f;
    for (int i = 0; i < nt >> 5; ++i) dot[j] += red[warp0 + i][j];
    s = fmaf(w[j], dot[j], s);
  }
  if (a.dw) {
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (tx == j && j < a.k) a.dw[t * a.k + j] = dot[j];
  }
  if (a.dlogits) {
    int id[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      id[j] = j < a.k ? a.ids[t * a.k + j] : -1;
      if (tx == 0 && j < a.k && (id[j] < 0 || id[j] >= a.E)) flag_status(status, MOE_ERR_INVALID_ARG);
    }
    for (int e = tx; e < a.E; e += nt) {
      float g = 0.f;
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (id[j] == e) g += w[j] * (dot[j] - s);
      a.dlogits[t * a.E + e] = g;
    }
  }
}

// Threads per token (a multiple of 32) and tokens per CTA.
dim3 rows_block(int nv) {
  int tx = 32;
  while (tx < nv && tx < kRowsThreads) tx *= 2;
  return dim3(tx, kRowsThreads / tx);
}

}  // namespace

#define MOE_ROWS(KERN)                                                                      \
  const int kb = a.k <= 1 ? 1 : (a.k <= 2 ? 2 : (a.k <= 4 ? 4 : 8));                        \
  auto kern = a.y_f32 ? KERN<8, true> : KERN<8, false>;                                     \
  if (kb == 4) kern = a.y_f32 ? KERN<4, true> : KERN<4, false>;                             \
  if (kb == 2) kern = a.y_f32 ? KERN<2, true> : KERN<2, false>;                             \
  if (kb == 1) kern = a.y_f32 ? KERN<1, true> : KERN<1, false>

cudaError_t launch_unpermute(const UnpermuteArgs& a, int* status, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  MOE_ROWS(unpermute_kernel);
  const int nv = a.H >> 3;
  const dim3 block = rows_block(nv);
  const dim3 grid((a.T + block.y - 1) / block.y, (nv + block.x - 1) / block.x);
  return launch_kernel(kern, grid, block, 0, st, a, status);
}

cudaError_t launch_unpermute_grad(const UnpermuteGradArgs& a, int* status, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  MOE_ROWS(unpermute_grad_kernel);
  const dim3 block = rows_block(a.H >> 3);
  return launch_kernel(kern, dim3((a.T + block.y - 1) / block.y), block, 0, st, a, status);
}
#undef MOE_ROWS

}  // namespace moe
