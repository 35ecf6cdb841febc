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
//   short rows (to 512 columns forward, 256 backward)  a warp per row, no barrier
//   longer rows              persistent CTAs, a row at a time: bulk copies bring
//                            the next rows to shared memory while the CTA takes
//                            one through its reductions
//   few rows (forward), rows above 8192 columns (backward): a CTA per row,
//                            straight from global memory
// Device time per call, inputs not in L2, and its share of the copy bandwidth (6794 GB/s):
//   rows   H     forward, bf16   backward, bf16, db and dres   rms_norm's, fp32 stream
//   8192   7168  46 us    75%    78 us    88%
//   2048   4096  9.8      50%    18.4     54%
//   16384  1024  17       58%    31       64%
//   16384  256   5.7      43%    12.5     40%
//   8192   4096                                                62 us   79%
//   16     4096  1.8      (launch and two reductions)  4.4 (two launches)        4.6
//   2047   5120                                                                24.5   63%
//   4096   12288 42       71%    150   39%                                     128    58%
//   2048   16384                 98    40%                                     82     60%
// The forward form is bound by instruction issue (62% of the slots), the backward
// one by DRAM on long rows and by latency on short ones: a CTA's threads take one row through its
// reduction with few others beside it (512 threads per SM at most, one CTA of 320 at 5120 columns).
// Rows above 8192 columns have no copies ahead, and 64 registers for two chunks per thread, which
// spill (216 bytes, rms_norm 40).  Short rows' forward grids are more CTAs than are resident, in rounds.
// The backward pass keeps a thread on the same columns for all of its rows and adds
// their part of dw and db in registers; each CTA leaves one row of partial sums,
// and a second kernel adds those in their order.
#include "block_tail.cuh"
#include "column_sum.cuh"
#include "common.cuh"
#include "norm_stages.h"
#include "tc_common.cuh"
#include "tc_ptx.cuh"
#include "train.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kNormThreads = 1024;
constexpr int kNarrowMaxV = 64;      // 8-column chunks of a row that a warp takes, forward
constexpr int kNarrowGradV = 32;     // and backward (16384 x 512: 25.2 us so, 21.7 streamed)
constexpr int kNarrowWarps = 8;      // rows at a time of a CTA then
constexpr int kNarrowCtas = 2;       // of them per SM, backward
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

// The sums of two values over the warp: the half-warps take one each after the first
// step.  Lanes 0 to 15 return v[0]'s, lanes 16 to 31 v[1]'s.
MOE_DEV float warp_halves(const float (&v)[2]) {
  const bool hi = (threadIdx.x & 16) != 0;
  float u = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  return u;
}

MOE_DEV void warp_sums2(float (&v)[2]) {
  const float u = warp_halves(v);
  v[0] = __shfl_sync(0xffffffffu, u, 0);
  v[1] = __shfl_sync(0xffffffffu, u, 16);
}

// Both over a CTA of at most 16 warps (red as in block_sums).
MOE_DEV void block_sums2(float (&v)[2], float (*red)[16]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float u = warp_halves(v);
  if ((lane & 15) == 0) red[lane >> 4][wid] = u;
  __syncthreads();
  if (nw > 1) {
    u = (lane & 15) < nw ? red[lane >> 4][lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  }
  v[0] = __shfl_sync(0xffffffffu, u, 0);
  v[1] = __shfl_sync(0xffffffffu, u, 16);
}

MOE_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

// The end of a CTA that streams rows; row n of the CTA goes to stage n % S.  Each thread
// waits for each row by itself, so a wait may run out in one and pass in another:
// whichever it was reports it.  Thread 0 sends for a stage again only after its own wait for
// the row before has passed, so where all of its waits have passed no copy is left; else the
// last one into each stage up to row `last` may be, and is waited for, with a limit, before
// the next CTA gets this shared memory.  (`last`, in shared memory, is written by thread 0 beside each
// copy: counting in a register took the forward pass of 8192 x 7168 from 46.1 to 48.1 us.)
MOE_DEV void stream_end(bool ok, uint64_t* full, int S, int64_t last, int* status) {
  if (ok) return;
  flag_status(status, MOE_ERR_TIMEOUT);
  if (threadIdx.x != 0) return;
  const int sent = (int)((last - blockIdx.x) / gridDim.x) + 1;
  uint32_t armed = 0, armed_ph = 0;
  for (int n = sent > S ? sent - S : 0; n < sent; ++n) {
    armed |= 1u << (n % S);
    armed_ph |= (uint32_t)((n / S) & 1) << (n % S);
  }
  tc::drain_armed(full, S, armed, armed_ph);
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
  MOE_DEV void get(float2 (&f)[4]) const {
    if constexpr (F32) {
      f[0] = make_float2(__uint_as_float(u[0].x), __uint_as_float(u[0].y));
      f[1] = make_float2(__uint_as_float(u[0].z), __uint_as_float(u[0].w));
      f[2] = make_float2(__uint_as_float(u[1].x), __uint_as_float(u[1].y));
      f[3] = make_float2(__uint_as_float(u[1].z), __uint_as_float(u[1].w));
    } else {
      f[0] = make_float2(bf16_lo(u[0].x), bf16_hi(u[0].x));
      f[1] = make_float2(bf16_lo(u[0].y), bf16_hi(u[0].y));
      f[2] = make_float2(bf16_lo(u[0].z), bf16_hi(u[0].z));
      f[3] = make_float2(bf16_lo(u[0].w), bf16_hi(u[0].w));
    }
  }
};

MOE_DEV void load_pairs(const void* p, bool f32, size_t at, float2 (&f)[4]) {
  if (f32) {
    Raw<true> r;
    r.load(p, at);
    r.get(f);
  } else {
    Raw<false> r;
    r.load(p, at);
    r.get(f);
  }
}

// The same from shared memory.
template <bool F32>
MOE_DEV Raw<F32> load_shared(uint32_t saddr) {
  Raw<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.u[i].x), "=r"(r.u[i].y), "=r"(r.u[i].z), "=r"(r.u[i].w)
                 : "r"(saddr + 16 * i));
  return r;
}

MOE_DEV void store_pairs(void* p, bool f32, size_t at, const float2 (&f)[4]) {
  const float v[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
  store8(p, f32, at, v);
}

MOE_DEV float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------ forward --
// What is left of a row once it is held in f (VPT chunks v0, v0 + step, ... per thread,
// zeros beyond the row): mean, centred squares, output.  sum adds one value over
// the row's threads; weights(i, v, w, b) gives a chunk's weight and bias.
template <int VPT, typename Sum, typename Weights>
MOE_DEV void layernorm_row(const LayerNormArgs& a, int64_t t, int v0, int step, float inv, float2 (&f)[VPT][4],
                           Sum sum, Weights weights) {
  const int nv = a.H >> 3;
  float2 s = both(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) s = add_f2(s, f[i][q]);
  const float mean = sum(s.x + s.y, 0) * inv;
  s = both(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (v0 + i * step < nv) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[i][q] = add_f2(f[i][q], both(-mean));
        s = fma_f2(f[i][q], f[i][q], s);
      }
    }
  const float rstd = rsqrtf(fmaf(sum(s.x + s.y, 1), inv, a.eps));  // (within two units in the last place)
  if (v0 == 0 && a.mean) {
    a.mean[t] = mean;
    a.rstd[t] = rstd;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= nv) continue;
    float2 w[4], b[4];
    weights(i, v, w, b);
#pragma unroll
    for (int q = 0; q < 4; ++q) f[i][q] = fma_f2(mul_f2(f[i][q], both(rstd)), w[q], b[q]);
    store_pairs(a.y, a.y_f32, (size_t)t * a.H + v * 8, f[i]);
  }
}

// The weights and bias of a thread's chunks for all of its rows: bf16 ones stay in
// registers, fp32 ones (and those of a thread with one row) are read where they are used.
template <int VPT, bool KEPT>
struct Weights {
  Raw<false> w[KEPT ? VPT : 1], b[KEPT ? VPT : 1];
  MOE_DEV void load(const LayerNormArgs& a, int v0, int step) {
    if constexpr (KEPT) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        b[i].zero();
        if (v0 + i * step < (a.H >> 3)) {
          w[i].load(a.w, (v0 + i * step) * 8);
          if (a.b) b[i].load(a.b, (v0 + i * step) * 8);
        }
      }
    }
  }
  MOE_DEV void get(const LayerNormArgs& a, int i, int v, float2 (&fw)[4], float2 (&fb)[4]) const {
    if constexpr (KEPT) {
      w[i].get(fw);
      b[i].get(fb);
    } else {
      load_pairs(a.w, a.w_f32, v * 8, fw);
#pragma unroll
      for (int q = 0; q < 4; ++q) fb[q] = both(0.f);
      if (a.b) load_pairs(a.b, a.w_f32, v * 8, fb);
    }
  }
};

// A warp takes the rows t, t + all warps, ...; the next one is on its way while it works
// on one.
template <int VPT, bool XF32, bool KEPT>
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
  Weights<VPT, KEPT> wb;
  wb.load(a, lane, 32);
  for (; t < a.T; t += step) {
    float2 f[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) next[i].get(f[i]);
    load(t + step);
    layernorm_row<VPT>(
        a, t, lane, 32, inv, f, [](float v, int) { return warp_sum(v); },
        [&](int i, int v, float2 (&w)[4], float2 (&b)[4]) { wb.get(a, i, v, w, b); });
  }
}

// CTA-wide forms: kRowVpt chunks per thread, so that the reductions' instructions, which every
// warp repeats, are few beside the row's own (8192 x 7168 bf16 with two chunks: 69 us).
constexpr int kRowNw = 32;

template <bool XF32, bool KEPT>
__global__ void __launch_bounds__(kRowNw * 32) layernorm_row_kernel(const LayerNormArgs a) {
  __shared__ float red[2][1][kRowNw];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x, nv = a.H >> 3;
  float2 f[kRowVpt][4];
#pragma unroll
  for (int i = 0; i < kRowVpt; ++i) {
    const int v = tid + i * nt;
#pragma unroll
    for (int q = 0; q < 4; ++q) f[i][q] = both(0.f);
    if (v < nv) load_pairs(a.x, XF32, (size_t)blockIdx.x * a.H + v * 8, f[i]);
  }
  Weights<kRowVpt, KEPT> wb;  // (on their way during the reductions)
  wb.load(a, tid, nt);
  layernorm_row<kRowVpt>(
      a, blockIdx.x, tid, nt, 1.0f / (float)a.H, f,
      [&](float v, int i) {
        float s[1] = {v};
        block_sums(s, red[i]);
        return s[0];
      },
      [&](int i, int v, float2 (&w)[4], float2 (&b)[4]) { wb.get(a, i, v, w, b); });
}

// Stage n % S holds row blockIdx.x + n gridDim.x.  A stage is free once the row's
// first reduction has passed (every thread holds its part), and thread 0 then sends for
// the row S further on.
template <bool XF32, bool KEPT>
__global__ void __launch_bounds__(kRowThreadsPerSm)
    layernorm_stream_kernel(const LayerNormArgs a, int S, int* status) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ float red[2][1][kRowNw];
  static_assert(sizeof(red) + kNormStages * 8 + 16 <= kCtaSmem - 1024, "the static part that the stages leave room for");
  __shared__ uint64_t full[kNormStages];
  __shared__ int s_abort;
  __shared__ int64_t s_last;  // row sent for last
  const int tid = threadIdx.x, nt = blockDim.x, nv = a.H >> 3;
  const float inv = 1.0f / (float)a.H;
  const uint32_t bytes = a.H * (XF32 ? 4 : 2);
  auto send = [&](int64_t t, int s) {
    s_last = t;
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
  Weights<kRowVpt, KEPT> wb;
  wb.load(a, tid, nt);
  int s = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    ok = ptx::mbar_wait(&full[s], ph, &s_abort) && ok;
    float2 f[kRowVpt][4];
#pragma unroll
    for (int i = 0; i < kRowVpt; ++i) {
      const int v = tid + i * nt;
#pragma unroll
      for (int q = 0; q < 4; ++q) f[i][q] = both(0.f);
      if (v < nv) load_shared<XF32>(ptx::smem_u32(stages) + s * bytes + v * (XF32 ? 32 : 16)).get(f[i]);
    }
    layernorm_row<kRowVpt>(
        a, t, tid, nt, inv, f,
        [&](float v, int i) {
          float r[1] = {v};
          block_sums(r, red[i]);
          if (i == 0 && tid == 0 && ok && t + (int64_t)S * gridDim.x < a.T) send(t + (int64_t)S * gridDim.x, s);
          return r[0];
        },
        [&](int i, int v, float2 (&w)[4], float2 (&b)[4]) { wb.get(a, i, v, w, b); });
    if (++s == S) {
      s = 0;
      ph ^= 1;
    }
  }
  stream_end(ok, full, S, s_last, status);
}

// ----------------------------------------------------------------- backward --
// One row, x and g = dy (VPT chunks per thread, zeros beyond the row); w(i, v, f) gives
// the weights of a chunk and res(i, v, f) its part of dres.  sum adds two values over the
// row's threads; store(at, f) writes a chunk of dx.
template <int VPT, bool RMS, typename Sum, typename W, typename Res, typename Store>
MOE_DEV void norm_grad_row(const NormGradArgs& a, int64_t t, int v0, int step, float inv, float2 (&x)[VPT][4],
                           float2 (&g)[VPT][4], float2 (&dw)[VPT][4], float2 (&db)[VPT][4], float m, float r, Sum sum,
                           W weights, Res res, Store store) {
  const int nv = a.H >> 3;
  float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= nv) continue;
    float2 w[4];
    weights(i, v, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 gw = mul_f2(g[i][q], w[q]);
      if (RMS) {
        s0 = fma_f2(x[i][q], x[i][q], s0);
      } else {
        x[i][q] = mul_f2(add_f2(x[i][q], both(-m)), both(r));
        s0 = add_f2(s0, gw);
      }
      s1 = fma_f2(gw, x[i][q], s1);
    }
  }
  float s[2] = {s0.x + s0.y, s1.x + s1.y};
  sum(s);
  float c0 = 0.f, c1 = s[1] * inv;
  if (RMS) {
    r = rsqrtf(fmaf(s[0], inv, a.eps));
    c1 *= r;
  } else {
    c0 = s[0] * inv;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= nv) continue;
    float2 w[4], d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = both(0.f);
    weights(i, v, w);
    if (a.dres) res(i, v, d);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 xh = RMS ? mul_f2(x[i][q], both(r)) : x[i][q];
      dw[i][q] = fma_f2(g[i][q], xh, dw[i][q]);
      if (!RMS) db[i][q] = add_f2(db[i][q], g[i][q]);
      d[q] = fma_f2(both(r), fma_f2(xh, both(-c1), fma_f2(g[i][q], w[q], both(-c0))), d[q]);
    }
    store((size_t)t * a.H + v * 8, d);
  }
}

// A thread's sums to the CTA's row [2, H] of the workspace.
template <int VPT>
MOE_DEV void norm_grad_part(const NormGradArgs& a, int v0, int step, const float2 (&dw)[VPT][4],
                            const float2 (&db)[VPT][4]) {
  float* part = static_cast<float*>(a.workspace) + (size_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * step;
    if (v >= (a.H >> 3)) continue;
    store_pairs(part, true, v * 8, dw[i]);
    if (a.db) store_pairs(part, true, a.H + v * 8, db[i]);
  }
}

template <int VPT, bool RMS, bool XF32, bool DF32>
__global__ void __launch_bounds__(kNarrowWarps * 32, kNarrowCtas) norm_grad_narrow_kernel(const NormGradArgs a) {
  __shared__ __align__(16) float sums[2][kNarrowGradV * 8];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nv = a.H >> 3;
  float2 dw[VPT][4] = {}, db[VPT][4] = {};
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
  const float inv = 1.0f / (float)a.H;
  float2 w[VPT][4] = {};
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (lane + i * 32 < nv) load_pairs(a.w, a.w_f32, (lane + i * 32) * 8, w[i]);
  for (; t < a.T; t += step) {
    float2 x[VPT][4], g[VPT][4];
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
        a, t, lane, 32, inv, x, g, dw, db, m, r, [](float (&s)[2]) { warp_sums2(s); },
        [&](int i, int, float2 (&e)[4]) {
#pragma unroll
          for (int q = 0; q < 4; ++q) e[q] = w[i][q];
        },
        [&](int i, int, float2 (&e)[4]) { d[i].get(e); },
        [&](size_t to, const float2 (&e)[4]) { store_pairs(a.dx, XF32, to, e); });
  }
  // the warps' sums, one warp after the other
  for (int k = 0; k < kNarrowWarps; ++k) {
    if (warp == k) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * 32;
        if (v >= nv) continue;
        float2* s0 = reinterpret_cast<float2*>(&sums[0][v * 8]);
        float2* s1 = reinterpret_cast<float2*>(&sums[1][v * 8]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (k > 0) {
            dw[i][q] = add_f2(s0[q], dw[i][q]);
            db[i][q] = add_f2(s1[q], db[i][q]);
          }
          s0[q] = dw[i][q];
          s1[q] = db[i][q];
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
  float2 dw[VPT][4] = {}, db[VPT][4] = {};
  int n = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, ++n) {
    const size_t at = (size_t)t * a.H;
    float2 x[VPT][4], g[VPT][4];
    float m = 0.f, r = 0.f;
    if (!RMS) {
      r = a.rstd[t];
      m = a.mean[t];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
#pragma unroll
      for (int q = 0; q < 4; ++q) x[i][q] = g[i][q] = both(0.f);
      if (v < nv) {
        load_pairs(a.x, a.x_f32, at + v * 8, x[i]);
        load_pairs(a.dy, a.dy_f32, at + v * 8, g[i]);
      }
    }
    norm_grad_row<VPT, RMS>(
        a, t, tid, nt, 1.0f / (float)a.H, x, g, dw, db, m, r, [&](float (&s)[2]) { block_sums(s, red[n & 1]); },
        [&](int, int v, float2 (&f)[4]) { load_pairs(a.w, a.w_f32, v * 8, f); },
        [&](int, int v, float2 (&d)[4]) { load_pairs(a.dres, a.x_f32, at + v * 8, d); },
        [&](size_t to, const float2 (&d)[4]) { store_pairs(a.dx, a.x_f32, to, d); });
  }
  norm_grad_part<VPT>(a, tid, nt, dw, db);
}

// The stages of layernorm_stream_kernel, each with the row's x, dy and dres.  The
// parts are in registers when the reduction has passed, so a stage is sent for again
// then.
template <bool RMS, bool XF32, bool DF32>
__global__ void __launch_bounds__(kGradNw * 32) norm_grad_stream_kernel(const NormGradArgs a, int S, int* status) {
  constexpr int V = kGradVpt;
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ float red[2][2][kGradNw];
  static_assert(sizeof(red) + kNormStages * 8 + 16 <= kCtaSmem - 1024, "the static part that the stages leave room for");
  __shared__ uint64_t full[kNormStages];
  __shared__ int s_abort;
  __shared__ int64_t s_last;  // row sent for last
  const int tid = threadIdx.x, nt = blockDim.x, nv = a.H >> 3;
  const uint32_t xb = a.H * (XF32 ? 4 : 2), gb = a.H * (DF32 ? 4 : 2), rb = a.dres ? xb : 0;
  const uint32_t stage = xb + gb + rb;
  auto send = [&](int64_t t, int s) {
    s_last = t;
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
  float2 dw[V][4] = {}, db[V][4] = {}, w[V][4] = {};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (tid + i * nt < nv) load_pairs(a.w, a.w_f32, (tid + i * nt) * 8, w[i]);
  const float inv = 1.0f / (float)a.H;
  float nm = 0.f, nr = 0.f;
  if (!RMS) {  // (the grid has no more CTAs than rows)
    nr = a.rstd[blockIdx.x];
    nm = a.mean[blockIdx.x];
  }
  int s = 0, n = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, ++n) {
    float2 x[V][4], g[V][4];
    Raw<XF32> d[V];
    const float m = nm, r = nr;
    if (!RMS && t + gridDim.x < a.T) {  // (a row ahead: their latency would be in every row)
      nr = a.rstd[t + gridDim.x];
      nm = a.mean[t + gridDim.x];
    }
    ok = ptx::mbar_wait(&full[s], ph, &s_abort) && ok;
    const uint32_t from = ptx::smem_u32(stages) + s * stage;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = tid + i * nt;
#pragma unroll
      for (int q = 0; q < 4; ++q) x[i][q] = g[i][q] = both(0.f);
      if (v < nv) {
        load_shared<XF32>(from + v * (XF32 ? 32 : 16)).get(x[i]);
        load_shared<DF32>(from + xb + v * (DF32 ? 32 : 16)).get(g[i]);
        if (rb) d[i] = load_shared<XF32>(from + xb + gb + v * (XF32 ? 32 : 16));
      }
    }
    norm_grad_row<V, RMS>(
        a, t, tid, nt, inv, x, g, dw, db, m, r,
        [&](float (&v)[2]) {
          block_sums2(v, red[n & 1]);
          if (tid == 0 && ok && t + (int64_t)S * gridDim.x < a.T) send(t + (int64_t)S * gridDim.x, s);
        },
        [&](int i, int, float2 (&f)[4]) {
#pragma unroll
          for (int q = 0; q < 4; ++q) f[q] = w[i][q];
        },
        [&](int i, int, float2 (&f)[4]) { d[i].get(f); },
        [&](size_t to, const float2 (&f)[4]) { store_pairs(a.dx, XF32, to, f); });
    if (++s == S) {
      s = 0;
      ph ^= 1;
    }
  }
  norm_grad_part<V>(a, tid, nt, dw, db);
  stream_end(ok, full, S, s_last, status);
}

// CTAs (rows of partial sums) of the backward pass on `sms` SMs.
int norm_grad_ctas(int T, int H, int sms) {
  const int nv = H >> 3;
  int64_t n, most;
  if (nv <= kNarrowGradV) {
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
    auto pick = [&](auto k) {
      constexpr bool K = decltype(k)::value;
      return nv <= 32 ? (a.x_f32 ? layernorm_narrow_kernel<1, true, K> : layernorm_narrow_kernel<1, false, K>)
                      : (a.x_f32 ? layernorm_narrow_kernel<2, true, K> : layernorm_narrow_kernel<2, false, K>);
    };
    auto kern = a.w_f32 ? pick(std::false_type{}) : pick(std::true_type{});
    return launch_kernel(kern, dim3(grid), dim3(kNarrowWarps * 32), 0, st, a);
  }
  const int threads = row_threads((nv + kRowVpt - 1) / kRowVpt), ctas = row_ctas(nv);
  const int64_t bytes = (int64_t)a.H * (a.x_f32 ? 4 : 2);
  if (a.T <= sms * ctas)
    return launch_kernel(
        a.x_f32 ? (a.w_f32 ? layernorm_row_kernel<true, false> : layernorm_row_kernel<true, true>)
                : (a.w_f32 ? layernorm_row_kernel<false, false> : layernorm_row_kernel<false, true>),
        dim3(a.T), dim3(threads), 0, st, a);
  const int S = norm_stages(ctas, bytes);
  auto kern = a.x_f32 ? (a.w_f32 ? layernorm_stream_kernel<true, false> : layernorm_stream_kernel<true, true>)
                      : (a.w_f32 ? layernorm_stream_kernel<false, false> : layernorm_stream_kernel<false, true>);
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
    if (nv <= kNarrowGradV) {
      auto pick = [&](auto x, auto d) {
        constexpr bool X = decltype(x)::value, D = decltype(d)::value;
        return rms ? norm_grad_narrow_kernel<1, true, X, D> : norm_grad_narrow_kernel<1, false, X, D>;
      };
      using T1 = std::true_type;
      using T0 = std::false_type;
      auto kern = a.x_f32 ? (a.dy_f32 ? pick(T1{}, T1{}) : pick(T1{}, T0{}))
                          : (a.dy_f32 ? pick(T0{}, T1{}) : pick(T0{}, T0{}));
      e = launch_kernel(kern, dim3(grid), dim3(kNarrowWarps * 32), 0, st, a);
    } else if (nv <= kGradVpt * kGradNw * 32) {
      const int threads = row_threads((nv + kGradVpt - 1) / kGradVpt);
      const int64_t bytes = (int64_t)a.H * ((a.x_f32 ? 4 : 2) * (a.dres ? 2 : 1) + (a.dy_f32 ? 4 : 2));
      const int S = norm_stages(grad_ctas(nv), bytes);
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
  return launch_column_sum((const float*)a.workspace, grid, 2 * (int64_t)a.H, cols, a.H, a.dw, a.db, sms, st);
}

}  // namespace moe
