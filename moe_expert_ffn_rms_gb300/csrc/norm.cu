// Layer norm forward and backward, and rms_norm's backward.
//
//   forward   mean = sum x / H, rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),
//             y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd, g = dy w,
//             dx = dres + rstd (g - sum g / H - xh sum(g xh) / H),
//             dw = sum_t dy xh, db = sum_t dy
//   rms_norm  mean = 0 and no sum of g: r = 1 / sqrt(sum x^2 / H + eps),
//             dx = dres + r (g - xh sum(g xh) / H), sum(g xh) = r sum(g x)
//
// Every row is read once and every result written once, so the bound is the
// copy bandwidth.  Statistics and sums are fp32.
#include "block_tail.cuh"
#include "common.cuh"
#include "train.h"

namespace moe {
namespace {

constexpr int kNormThreads = 1024;

// Sums of N values over the CTA; every thread gets them.  `red` is N x 32 floats
// that nothing else uses until the next __syncthreads.
template <int N>
MOE_DEV void block_sums(float (&v)[N], float (*red)[32]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = warp_sum(v[i]);
    if (lane == 0) red[i][wid] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < nw ? red[i][lane] : 0.f);
}

// One CTA per row, held in registers: VPT chunks of 8 columns per thread.
template <int VPT>
__global__ void __launch_bounds__(kNormThreads) layernorm_kernel(const LayerNormArgs a) {
  __shared__ float red[2][1][32];
  pdl_trigger();
  pdl_wait();
  const size_t at = (size_t)blockIdx.x * a.H;
  const int nv = a.H >> 3, tid = threadIdx.x, nt = blockDim.x;
  float f[VPT][8], s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * nt;
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
    if (v < nv) load8(a.x, a.x_f32, at + v * 8, f[i]);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) s[0] += f[i][q];
  block_sums(s, red[0]);
  const float mean = s[0] / (float)a.H;
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (tid + i * nt < nv) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[i][q] -= mean;
        s[0] = fmaf(f[i][q], f[i][q], s[0]);
      }
    }
  block_sums(s, red[1]);
  const float rstd = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
  if (tid == 0 && a.mean) {
    a.mean[blockIdx.x] = mean;
    a.rstd[blockIdx.x] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * nt;
    if (v >= nv) continue;
    float w[8], b[8] = {};
    load8(a.w, a.w_f32, v * 8, w);
    if (a.b) load8(a.b, a.w_f32, v * 8, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = fmaf(f[i][q] * rstd, w[q], b[q]);
    store8(a.y, a.y_f32, at + v * 8, f[i]);
  }
}

// ----------------------------------------------------------------- backward --
// CTA c takes rows c, c + grid, ...; a thread keeps the same columns for all of
// them and adds their part of dw and db in registers, written to the workspace
// as row c of [grid, 2, H] at the end and summed by norm_grad_sum_kernel.
template <int VPT, bool RMS>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float red[2][2][32];
  pdl_trigger();
  pdl_wait();
  const int nv = a.H >> 3, tid = threadIdx.x, nt = blockDim.x;
  const float inv = 1.0f / (float)a.H;
  float dw[VPT][8] = {}, db[VPT][8] = {};
  int n = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, ++n) {
    const size_t at = (size_t)t * a.H;
    float r = 0.f, m = 0.f;
    if (!RMS) {
      r = a.rstd[t];
      m = a.mean[t];
    }
    float x[VPT][8], g[VPT][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[i][q] = g[i][q] = 0.f;
      if (v < nv) {
        load8(a.x, a.x_f32, at + v * 8, x[i]);
        load8(a.dy, a.dy_f32, at + v * 8, g[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
      if (v >= nv) continue;
      float w[8];
      load8(a.w, a.w_f32, v * 8, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float gw = g[i][q] * w[q];
        if (RMS) {
          s[0] = fmaf(x[i][q], x[i][q], s[0]);
        } else {
          x[i][q] = (x[i][q] - m) * r;
          s[0] += gw;
        }
        s[1] = fmaf(gw, x[i][q], s[1]);
      }
    }
    block_sums(s, red[n & 1]);
    float c0 = 0.f, c1;
    if (RMS) {
      r = 1.0f / sqrtf(s[0] * inv + a.eps);
      c1 = s[1] * r * inv;
    } else {
      c0 = s[0] * inv;
      c1 = s[1] * inv;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
      if (v >= nv) continue;
      float w[8], d[8] = {};
      load8(a.w, a.w_f32, v * 8, w);
      if (a.dres) load8(a.dres, a.x_f32, at + v * 8, d);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xh = RMS ? x[i][q] * r : x[i][q];
        dw[i][q] = fmaf(g[i][q], xh, dw[i][q]);
        if (!RMS) db[i][q] += g[i][q];
        d[q] = fmaf(r, fmaf(g[i][q], w[q], -c0) - xh * c1, d[q]);
      }
      store8(a.dx, a.x_f32, at + v * 8, d);
    }
  }
  float* part = static_cast<float*>(a.workspace) + (size_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * nt;
    if (v >= nv) continue;
    store8(part, true, v * 8, dw[i]);
    if (a.db) store8(part, true, a.H + v * 8, db[i]);
  }
}

// dw (and db) = the sum of the n partial rows, in their order.
__global__ void __launch_bounds__(256) norm_grad_sum_kernel(const float* __restrict__ part, int n, int H,
                                                            float* dw, float* db) {
  __shared__ float red[8][32];
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
  float s = 0.f;
  if (c < (db ? 2 * H : H))
    for (int i = y; i < n; i += 8) s += part[(size_t)i * 2 * H + c];
  red[y][threadIdx.x & 31] = s;
  __syncthreads();
  if (y != 0 || c >= (db ? 2 * H : H)) return;
  for (int i = 1; i < 8; ++i) s += red[i][threadIdx.x];
  if (c < H) dw[c] = s;
  else db[c - H] = s;
}

constexpr int kGradRows = 304;  // partial rows at most

}  // namespace

cudaError_t launch_layernorm(const LayerNormArgs& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const int nv = a.H >> 3;
  const int vpt = nv <= 256 ? 1 : 2;
  const int threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
  return launch_kernel(vpt == 1 ? layernorm_kernel<1> : layernorm_kernel<2>, dim3(a.T), dim3(threads), 0, st,
                       a);
}

size_t norm_grad_workspace_bytes(int T, int H) {
  return (size_t)(T < kGradRows ? T : kGradRows) * 2 * H * sizeof(float);
}

cudaError_t launch_norm_grad(const NormGradArgs& a, int sms, int* status, cudaStream_t st) {
  const int nv = a.H >> 3;
  const int vpt = nv <= 256 ? 1 : 2;
  const int threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
  int grid = threads <= 512 ? 2 * sms : sms;
  if (grid > a.T) grid = a.T;
  if (grid > kGradRows) grid = kGradRows;
  if (grid > 0) {
    auto kern = vpt == 1 ? norm_grad_kernel<1, false> : norm_grad_kernel<2, false>;
    if (!a.mean) kern = vpt == 1 ? norm_grad_kernel<1, true> : norm_grad_kernel<2, true>;
    cudaError_t e = launch_kernel(kern, dim3(grid), dim3(threads), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  const int cols = a.db ? 2 * a.H : a.H;
  return launch_kernel(norm_grad_sum_kernel, dim3((cols + 31) / 32), dim3(256), 0, st,
                       (const float*)a.workspace, grid, a.H, a.dw, a.db);
}

}  // namespace moe
