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
// copy bandwidth.  Statistics and sums are fp32.  Three forms:
//   rows up to 512 columns   a warp per row, no barrier
//   longer rows              persistent CTAs, a row at a time: bulk copies bring
//                            the next rows to shared memory while the CTA takes
//                            one through its reductions
//   few rows (forward), rows above 8192 columns (backward): a CTA per row,
//                            straight from global memory
// The backward pass keeps a thread on the same columns for all of its rows and adds
// their part of dw and db in registers; each CTA leaves one row of partial sums,
// and a second kernel adds those in their order.
#include "block_tail.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"
#include "train.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kNormThreads = 1024;
constexpr int kNarrowMaxV = 64;      // 8-column chunks of a row that a warp takes
constexpr int kNarrowWarps = 8;      // rows at a time of a CTA then
constexpr int kNarrowCtas = 2;       // of them per SM, backward
constexpr int kNormStages = 8;       // rows on their way at most
constexpr int kNormSmem = 212 << 10; // per SM, for the stages
constexpr int kMaxSms = 160;         // the workspace's size goes by it

// Sums of N values over the CTA of at most NW warps; every thread gets them.  `red` is
// not used by anything else until the next __syncthreads.
template <int NW, int N>
MOE_DEV void block_sums(float (&v)[N], float (*red)[NW]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][wid] = v[i];
  }
  __syncthreads();
  if (nw == 1) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float u = (lane & (NW - 1)) < nw ? red[i][lane & (NW - 1)] : 0.f;
#pragma unroll
    for (int o = NW / 2; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    v[i] = u;
  }
}

template <int N>
MOE_DEV void warp_sums(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
}

MOE_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ forward --
// What is left of a row once it is held in f (VPT chunks v0, v0 + step, ... per thread,
// zeros beyond the row): mean, centred squares, output.  SUM adds one value over
// the row's threads.
template <int VPT, typename Sum>
MOE_DEV void layernorm_row(const LayerNormArgs& a, int64_t t, int v0, int step, float inv, float (&f)[VPT][8],
                           Sum sum) {
  const int nv = a.H >> 3;
  const size_t at = (size_t)t * a.H;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) s += f[i][q];
  const float mean = sum(s, 0) * inv;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (v0 + i * step < nv) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[i][q] -= mean;
        s = fmaf(f[i][q], f[i][q], s);
      }
    }
  const float rstd = 1.0f / sqrtf(fmaf(sum(s, 1), inv, a.eps));
  if (v0 == 0 && a.mean) {
    a.mean[t] = mean;
    a.rstd[t] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= nv) continue;
    float w[8], b[8] = {};
    load8(a.w, a.w_f32, v * 8, w);
    if (a.b) load8(a.b, a.w_f32, v * 8, b);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = fmaf(f[i][q] * rstd, w[q], b[q]);
    store8(a.y, a.y_f32, at + v * 8, f[i]);
  }
}

// Eight columns as they are in memory.
template <bool F32>
struct Raw {
  uint4 u[F32 ? 2 : 1];
  MOE_DEV void load(const void* p, size_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) u[i] = s[i];
  }
  MOE_DEV void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  MOE_DEV void get(float (&f)[8]) const {
    if constexpr (F32) {
      f[0] = __uint_as_float(u[0].x); f[1] = __uint_as_float(u[0].y);
      f[2] = __uint_as_float(u[0].z); f[3] = __uint_as_float(u[0].w);
      f[4] = __uint_as_float(u[1].x); f[5] = __uint_as_float(u[1].y);
      f[6] = __uint_as_float(u[1].z); f[7] = __uint_as_float(u[1].w);
    } else {
      unpack8_bf16(u[0], f);
    }
  }
};

// A warp takes the rows t, t + all warps, ...; the next one is on its way while it works
// on one.
template <int VPT, bool XF32>
__global__ void __launch_bounds__(kNarrowWarps * 32) layernorm_narrow_kernel(const LayerNormArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, nv = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  const int64_t step = (int64_t)gridDim.x * kNarrowWarps;
  int64_t t = (int64_t)blockIdx.x * kNarrowWarps + (threadIdx.x >> 5);
  Raw<XF32> next[VPT];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      next[i].zero();
      if (row < a.T && lane + i * 32 < nv) next[i].load(a.x, (size_t)row * a.H + (lane + i * 32) * 8);
    }
  };
  load(t);
  for (; t < a.T; t += step) {
    float f[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) next[i].get(f[i]);
    load(t + step);
    layernorm_row<VPT>(a, t, lane, 32, inv, f, [](float v, int) { return warp_sum(v); });
  }
}

// CTA-wide forms: kRowVpt chunks per thread, so that the reductions' instructions, which every
// warp repeats, are few beside the row's own (8192 x 7168 bf16 with two chunks: 69 us).
constexpr int kRowVpt = 4;
constexpr int kRowNw = 16;

template <bool XF32>
__global__ void __launch_bounds__(kRowNw * 32) layernorm_row_kernel(const LayerNormArgs a) {
  __shared__ float red[2][1][kRowNw];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x, nv = a.H >> 3;
  float f[kRowVpt][8];
#pragma unroll
  for (int i = 0; i < kRowVpt; ++i) {
    const int v = tid + i * nt;
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
    if (v < nv) load8(a.x, XF32, (size_t)blockIdx.x * a.H + v * 8, f[i]);
  }
  layernorm_row<kRowVpt>(a, blockIdx.x, tid, nt, 1.0f / (float)a.H, f, [&](float v, int i) {
    float s[1] = {v};
    block_sums(s, red[i]);
    return s[0];
  });
}

// Stage n % S holds row blockIdx.x + n gridDim.x.  A stage is free once the row's
// first reduction has passed (every thread holds its part), and thread 0 then sends for
// the row S further on.
template <bool XF32>
__global__ void __launch_bounds__(kRowNw * 32, 2)
    layernorm_stream_kernel(const LayerNormArgs a, int S, int* status) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ float red[2][1][kRowNw];
  __shared__ uint64_t full[kNormStages];
  __shared__ int s_abort;
  const int tid = threadIdx.x, nt = blockDim.x, nv = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  const uint32_t bytes = a.H * (XF32 ? 4 : 2);
  auto send = [&](int64_t t, int s) {
    ptx::mbar_arrive_expect_tx(&full[s], bytes);
    bulk_load(stages + (size_t)s * bytes, static_cast<const unsigned char*>(a.x) + (size_t)t * bytes, bytes, &full[s]);
  };
  pdl_trigger();
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < S; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  if (tid == 0)
    for (int s = 0; s < S; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < a.T) send(blockIdx.x + (int64_t)s * gridDim.x, s);
  int s = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    ok = ptx::mbar_wait(&full[s], ph, &s_abort) && ok;
    float f[kRowVpt][8];
#pragma unroll
    for (int i = 0; i < kRowVpt; ++i) {
      const int v = tid + i * nt;
#pragma unroll
      for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
      if (v < nv) load8(stages + (size_t)s * bytes, XF32, v * 8, f[i]);
    }
    layernorm_row<kRowVpt>(a, t, tid, nt, inv, f, [&](float v, int i) {
      float r[1] = {v};
      block_sums(r, red[i]);
      if (i == 0 && tid == 0 && ok && t + (int64_t)S * gridDim.x < a.T) send(t + (int64_t)S * gridDim.x, s);
      return r[0];
    });
    if (++s == S) {
      s = 0;
      ph ^= 1;
    }
  }
  if (!ok && tid == 0) flag_status(status, MOE_ERR_TIMEOUT);
}

// ----------------------------------------------------------------- backward --
// One row, x and g = dy (VPT chunks per thread, zeros beyond the row) and res(i, v, d)
// to load dres's chunk.  sum adds two values over the row's threads.
template <int VPT, bool RMS, typename Sum, typename Res>
MOE_DEV void norm_grad_row(const NormGradArgs& a, int64_t t, int v0, int step, float (&x)[VPT][8],
                           float (&g)[VPT][8], float (&dw)[VPT][8], float (&db)[VPT][8], float m, float r, Sum sum,
                           Res res) {
  const int nv = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
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
  sum(s);
  float c0 = 0.f, c1 = s[1] * inv;
  if (RMS) {
    r = 1.0f / sqrtf(fmaf(s[0], inv, a.eps));
    c1 *= r;
  } else {
    c0 = s[0] * inv;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= nv) continue;
    float w[8], d[8] = {};
    load8(a.w, a.w_f32, v * 8, w);
    if (a.dres) res(i, v, d);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float xh = RMS ? x[i][q] * r : x[i][q];
      dw[i][q] = fmaf(g[i][q], xh, dw[i][q]);
      if (!RMS) db[i][q] += g[i][q];
      d[q] = fmaf(r, fmaf(g[i][q], w[q], -c0) - xh * c1, d[q]);
    }
    store8(a.dx, a.x_f32, (size_t)t * a.H + v * 8, d);
  }
}

// A thread's sums to the CTA's row [2, H] of the workspace.
template <int VPT>
MOE_DEV void norm_grad_part(const NormGradArgs& a, int v0, int step, const float (&dw)[VPT][8],
                            const float (&db)[VPT][8]) {
  float* part = static_cast<float*>(a.workspace) + (size_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= (a.H >> 3)) continue;
    store8(part, true, v * 8, dw[i]);
    if (a.db) store8(part, true, a.H + v * 8, db[i]);
  }
}

template <int VPT, bool RMS, bool XF32, bool DF32>
__global__ void __launch_bounds__(kNarrowWarps * 32, kNarrowCtas) norm_grad_narrow_kernel(const NormGradArgs a) {
  __shared__ float sums[2][kNarrowMaxV * 8];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nv = a.H >> 3;
  float dw[VPT][8] = {}, db[VPT][8] = {};
  const int64_t step = (int64_t)gridDim.x * kNarrowWarps;
  int64_t t = (int64_t)blockIdx.x * kNarrowWarps + warp;
  Raw<XF32> nx[VPT], nd[VPT];
  Raw<DF32> ng[VPT];
  float nm = 0.f, nr = 0.f;
  auto load = [&](int64_t row) {  // the next row, while the warp works on one
    if (!RMS && row < a.T) {
      nr = a.rstd[row];
      nm = a.mean[row];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const size_t at = (size_t)row * a.H + (lane + i * 32) * 8;
      nx[i].zero();
      ng[i].zero();
      if (row < a.T && lane + i * 32 < nv) {
        nx[i].load(a.x, at);
        ng[i].load(a.dy, at);
        if (a.dres) nd[i].load(a.dres, at);
      }
    }
  };
  load(t);
  for (; t < a.T; t += step) {
    float x[VPT][8], g[VPT][8];
    Raw<XF32> d[VPT];
    const float m = nm, r = nr;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      nx[i].get(x[i]);
      ng[i].get(g[i]);
      d[i] = nd[i];
    }
    load(t + step);
    norm_grad_row<VPT, RMS>(
        a, t, lane, 32, x, g, dw, db, m, r, [](float (&s)[2]) { warp_sums(s); },
        [&](int i, int, float (&e)[8]) { d[i].get(e); });
  }
  // the warps' sums, one warp after the other
  for (int k = 0; k < kNarrowWarps; ++k) {
    if (warp == k) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * 32;
        if (v >= nv) continue;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (k > 0) {
            dw[i][q] += sums[0][v * 8 + q];
            db[i][q] += sums[1][v * 8 + q];
          }
          sums[0][v * 8 + q] = dw[i][q];
          sums[1][v * 8 + q] = db[i][q];
        }
      }
    }
    __syncthreads();
  }
  if (warp == kNarrowWarps - 1) norm_grad_part<VPT>(a, lane, 32, dw, db);
}

template <int VPT, bool RMS>
__global__ void __launch_bounds__(kNormThreads) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float red[2][2][32];
  pdl_trigger();
  pdl_wait();
  const int nv = a.H >> 3, tid = threadIdx.x, nt = blockDim.x;
  float dw[VPT][8] = {}, db[VPT][8] = {};
  int n = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, ++n) {
    const size_t at = (size_t)t * a.H;
    float x[VPT][8], g[VPT][8], m = 0.f, r = 0.f;
    if (!RMS) {
      r = a.rstd[t];
      m = a.mean[t];
    }
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
    norm_grad_row<VPT, RMS>(
        a, t, tid, nt, x, g, dw, db, m, r, [&](float (&s)[2]) { block_sums(s, red[n & 1]); },
        [&](int, int v, float (&d)[8]) { load8(a.dres, a.x_f32, at + v * 8, d); });
  }
  norm_grad_part<VPT>(a, tid, nt, dw, db);
}

constexpr int kGradVpt = 2;
constexpr int kGradNw = 16;

// The stages of layernorm_stream_kernel, each with the row's x, dy and dres.  The
// parts are in registers when the reduction has passed, so a stage is sent for again
// then.
template <bool RMS, bool XF32, bool DF32>
__global__ void __launch_bounds__(kGradNw * 32) norm_grad_stream_kernel(const NormGradArgs a, int S, int* status) {
  constexpr int V = kGradVpt;
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ float red[2][2][kGradNw];
  __shared__ uint64_t full[kNormStages];
  __shared__ int s_abort;
  const int tid = threadIdx.x, nt = blockDim.x, nv = a.H >> 3;
  const uint32_t xb = a.H * (XF32 ? 4 : 2), gb = a.H * (DF32 ? 4 : 2), rb = a.dres ? xb : 0;
  const uint32_t stage = xb + gb + rb;
  auto send = [&](int64_t t, int s) {
    unsigned char* to = stages + (size_t)s * stage;
    ptx::mbar_arrive_expect_tx(&full[s], stage);
    bulk_load(to, static_cast<const unsigned char*>(a.x) + (size_t)t * xb, xb, &full[s]);
    bulk_load(to + xb, static_cast<const unsigned char*>(a.dy) + (size_t)t * gb, gb, &full[s]);
    if (rb) bulk_load(to + xb + gb, static_cast<const unsigned char*>(a.dres) + (size_t)t * rb, rb, &full[s]);
  };
  pdl_trigger();
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < S; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  if (tid == 0)
    for (int s = 0; s < S; ++s)
      if (blockIdx.x + (int64_t)s * gridDim.x < a.T) send(blockIdx.x + (int64_t)s * gridDim.x, s);
  float dw[V][8] = {}, db[V][8] = {};
  int s = 0, n = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, ++n) {
    float x[V][8], g[V][8], m = 0.f, r = 0.f;
    Raw<XF32> d[V];
    if (!RMS) {
      r = a.rstd[t];
      m = a.mean[t];
    }
    ok = ptx::mbar_wait(&full[s], ph, &s_abort) && ok;
    const unsigned char* from = stages + (size_t)s * stage;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * nt;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[i][q] = g[i][q] = 0.f;
      if (v < nv) {
        load8(from, XF32, v * 8, x[i]);
        load8(from + xb, DF32, v * 8, g[i]);
        if (rb) d[i].load(from + xb + gb, v * 8);
      }
    }
    norm_grad_row<V, RMS>(
        a, t, tid, nt, x, g, dw, db, m, r,
        [&](float (&v)[2]) {
          block_sums(v, red[n & 1]);
          if (tid == 0 && ok && t + (int64_t)S * gridDim.x < a.T) send(t + (int64_t)S * gridDim.x, s);
        },
        [&](int i, int, float (&e)[8]) { d[i].get(e); });
    if (++s == S) {
      s = 0;
      ph ^= 1;
    }
  }
  norm_grad_part<V>(a, tid, nt, dw, db);
  if (!ok && tid == 0) flag_status(status, MOE_ERR_TIMEOUT);
}

// dw (and db) = the sum of the n partial rows, in their order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_grad_sum_kernel(const float* __restrict__ part, int n, int H,
                                                                       float* dw, float* db) {
  __shared__ float red[kSumWarps][32];
  pdl_trigger();
  pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, cols = db ? 2 * H : H;
  const int c = blockIdx.x * 32 + x;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int i = y; i < n; i += kSumWarps) s += part[(size_t)i * 2 * H + c];
  }
  red[y][x] = s;
  __syncthreads();
  if (y != 0 || c >= cols) return;
  for (int i = 1; i < kSumWarps; ++i) s += red[i][x];
  if (c < H) dw[c] = s;
  else db[c - H] = s;
}

int row_threads(int nv) { return (nv + 31) / 32 * 32; }

// CTAs per SM: the forward kernels are held to 64 registers, the backward ones to 128.
int row_ctas(int nv) {
  const int n = 1024 / row_threads((nv + kRowVpt - 1) / kRowVpt);
  return n < 16 ? n : 16;
}
int grad_ctas(int nv) {
  const int n = 512 / row_threads((nv + kGradVpt - 1) / kGradVpt);
  return n < 8 ? n : 8;
}

// CTAs (rows of partial sums) of the backward pass on `sms` SMs.
int norm_grad_ctas(int T, int H, int sms) {
  const int nv = H >> 3;
  int64_t n, most;
  if (nv <= kNarrowMaxV) {
    n = ((int64_t)T + kNarrowWarps - 1) / kNarrowWarps;
    most = (int64_t)sms * kNarrowCtas;
  } else {
    n = T;
    most = (int64_t)sms * (nv <= kGradVpt * kGradNw * 32 ? grad_ctas(nv) : 1);
  }
  return (int)(n < most ? n : most);
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormArgs& a, int sms, int* status, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const int nv = a.H >> 3;
  if (nv <= kNarrowMaxV) {
    const int64_t n = ((int64_t)a.T + kNarrowWarps - 1) / kNarrowWarps;
    const int grid = (int)(n < sms * 8 ? n : sms * 8);
    auto kern = nv <= 32 ? (a.x_f32 ? layernorm_narrow_kernel<1, true> : layernorm_narrow_kernel<1, false>)
                         : (a.x_f32 ? layernorm_narrow_kernel<2, true> : layernorm_narrow_kernel<2, false>);
    return launch_kernel(kern, dim3(grid), dim3(kNarrowWarps * 32), 0, st, a);
  }
  const int threads = row_threads((nv + kRowVpt - 1) / kRowVpt), ctas = row_ctas(nv);
  const int64_t bytes = (int64_t)a.H * (a.x_f32 ? 4 : 2);
  if (a.T <= sms * ctas)
    return launch_kernel(a.x_f32 ? layernorm_row_kernel<true> : layernorm_row_kernel<false>, dim3(a.T), dim3(threads),
                         0, st, a);
  int S = (int)(kNormSmem / ctas / bytes);
  if (S > kNormStages) S = kNormStages;
  auto kern = a.x_f32 ? layernorm_stream_kernel<true> : layernorm_stream_kernel<false>;
  // the same limit in every call: another thread's launch may lie between this and ours
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(sms * ctas), dim3(threads), (size_t)S * bytes, st, a, S, status);
}

size_t norm_grad_workspace_bytes(int T, int H) {
  return (size_t)norm_grad_ctas(T, H, kMaxSms) * 2 * H * sizeof(float);
}

cudaError_t launch_norm_grad(const NormGradArgs& a, int sms, int* status, cudaStream_t st) {
  const int nv = a.H >> 3;
  const int grid = norm_grad_ctas(a.T, a.H, sms < kMaxSms ? sms : kMaxSms);
  const bool rms = !a.mean;
  if (grid > 0) {
    cudaError_t e;
    if (nv <= kNarrowMaxV) {
      auto pick = [&](auto x, auto d) {
        constexpr bool X = decltype(x)::value, D = decltype(d)::value;
        if (nv <= 32) return rms ? norm_grad_narrow_kernel<1, true, X, D> : norm_grad_narrow_kernel<1, false, X, D>;
        return rms ? norm_grad_narrow_kernel<2, true, X, D> : norm_grad_narrow_kernel<2, false, X, D>;
      };
      using T1 = std::true_type;
      using T0 = std::false_type;
      auto kern = a.x_f32 ? (a.dy_f32 ? pick(T1{}, T1{}) : pick(T1{}, T0{}))
                          : (a.dy_f32 ? pick(T0{}, T1{}) : pick(T0{}, T0{}));
      e = launch_kernel(kern, dim3(grid), dim3(kNarrowWarps * 32), 0, st, a);
    } else if (nv <= kGradVpt * kGradNw * 32) {
      const int threads = row_threads((nv + kGradVpt - 1) / kGradVpt);
      const int64_t bytes = (int64_t)a.H * ((a.x_f32 ? 4 : 2) * (a.dres ? 2 : 1) + (a.dy_f32 ? 4 : 2));
      int S = (int)(kNormSmem / grad_ctas(nv) / bytes);
      if (S > kNormStages) S = kNormStages;
      auto pick = [&](auto r) {
        constexpr bool R = decltype(r)::value;
        return a.x_f32 ? (a.dy_f32 ? norm_grad_stream_kernel<R, true, true> : norm_grad_stream_kernel<R, true, false>)
                       : (a.dy_f32 ? norm_grad_stream_kernel<R, false, true> : norm_grad_stream_kernel<R, false, false>);
      };
      auto kern = rms ? pick(std::true_type{}) : pick(std::false_type{});
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
      if (e == cudaSuccess)
        e = launch_kernel(kern, dim3(grid), dim3(threads), (size_t)S * bytes, st, a, S, status);
    } else {
      const int threads = row_threads((nv + 1) / 2);
      e = launch_kernel(rms ? norm_grad_kernel<2, true> : norm_grad_kernel<2, false>, dim3(grid), dim3(threads), 0, st, a);
    }
    if (e != cudaSuccess) return e;
  }
  const int cols = a.db ? 2 * a.H : a.H;
  return launch_kernel(norm_grad_sum_kernel, dim3((cols + 31) / 32), dim3(kSumWarps * 32), 0, st,
                       (const float*)a.workspace, grid, a.H, a.dw, a.db);
}

}  // namespace moe
