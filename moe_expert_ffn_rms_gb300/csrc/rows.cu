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
// copy bandwidth (6794 GB/s measured).  Device time per call, inputs not in L2, bf16:
//   T    H    k     return, residual       gradient with the router's
//   4096 4096 8     53.3 us    93%         92 us   91%
//   8192 2048 4     33.4       89%         53      83%
//   8192 512  8     15.8       78%         31      68%
//   4096 4096 8     89.6       99%         169     96%      (fp32 expert rows)
//   64   4096 8                            5.8     (launch, two dependent loads, a reduction)
//   1    4096 8      1.9                   4.1
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

// 16 bytes that are read once: kept out of L1.
MOE_DEV uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

constexpr int kRowsThreads = 256;  // of a CTA at most

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
      for (int i = 0; i < W; ++i) q[j][i] = load_once(s + i);
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

// blockDim.x lanes take PP consecutive slots of a token, so each row's dot product stays with
// its warps and dout's row is loaded once for them; the slots of a token lie in one CTA
// (blockDim.y = groups of slots x tokens).  N chunks of dout and of each slot's row are in
// flight per lane: four with one slot, two of fp32 or with four slots (short rows, of which a
// lane has no more: T = 8192, H = 512, k = 8 45.2 us with one).
// (A CTA per token with all k rows in flight per thread, at T = 4096, H = 4096, k = 8:
// 123 registers, 113 us; so 91.)
constexpr int kGradThreads = 1024;

// Eight columns as they are in memory.
template <bool F32>
struct Raw {
  uint4 u[F32 ? 2 : 1];
  MOE_DEV void load(const void* p, size_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) u[i] = s[i];
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

template <bool YF32, bool DF32, int N, int PP>
__global__ void __launch_bounds__(PP == 1 ? kGradThreads : 256) unpermute_grad_kernel(const UnpermuteGradArgs a, int groups,
                                                                      int* status) {
  __shared__ float red[kGradThreads / 32][PP];
  __shared__ float s_dw[kGradThreads / 32][kMaxTopK], s_w[kGradThreads / 32][kMaxTopK];
  __shared__ int s_id[kGradThreads / 32][kMaxTopK];
  pdl_trigger();
  pdl_wait();
  const int nv = a.H >> 3, tx = threadIdx.x, ty = threadIdx.y, nt = blockDim.x;
  const int local = ty / groups, group = ty - local * groups, j0 = group * PP;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.y / groups) + local;
  const bool on = t < a.T;
  const bool dots = a.dw || a.dlogits;
  const size_t at_d = (size_t)t * a.H;
  Raw<DF32> d[N];
  auto load_dout = [&](int v0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (v0 + i * nt < nv) d[i].load(a.dout, at_d + (v0 + i * nt) * 8);
  };
  int row[PP], id[PP];
  float w[PP], dot[PP];
  bool any = false;
#pragma unroll
  for (int p = 0; p < PP; ++p) {
    row[p] = id[p] = -1;
    w[p] = dot[p] = 0.f;
  }
  if (on) {
    load_dout(tx);  // (does not wait for the rows' indices)
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      if (j0 + p < a.k) {
        const int64_t pair = t * a.k + j0 + p;
        row[p] = pair_row(a.row_of_pair, pair, a.T * a.k, tx == 0, status);
        w[p] = a.w[pair];
        if (a.dlogits && tx == 0) id[p] = a.ids[pair];
        any |= row[p] >= 0;
      }
    }
  }
  if (any) {
    for (int v0 = tx; v0 < nv; v0 += nt * N) {
      Raw<YF32> y[PP][N];
      if (dots) {
#pragma unroll
        for (int p = 0; p < PP; ++p)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (row[p] >= 0 && v0 + i * nt < nv) y[p][i].load(a.y, (size_t)row[p] * a.H + (v0 + i * nt) * 8);
      }
      if (v0 != tx) load_dout(v0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = v0 + i * nt;
        if (v >= nv) break;
        float f[8];
        d[i].get(f);
#pragma unroll
        for (int p = 0; p < PP; ++p) {
          if (row[p] < 0) continue;
          if (dots) {
            float g[8];
            y[p][i].get(g);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[p] = fmaf(f[q], g[q], dot[p]);
          }
          if (a.dy) {
            float g[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) g[q] = f[q] * w[p];
            store8(a.dy, YF32, (size_t)row[p] * a.H + v * 8, g);
          }
        }
      }
    }
  }
  if (!dots) return;
#pragma unroll
  for (int p = 0; p < PP; ++p) dot[p] = warp_sum(dot[p]);
  const int wp = nt >> 5;
  if (wp > 1) {
    if ((tx & 31) == 0) {
#pragma unroll
      for (int p = 0; p < PP; ++p) red[ty * wp + (tx >> 5)][p] = dot[p];
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      dot[p] = 0.f;
      for (int i = 0; i < wp; ++i) dot[p] += red[ty * wp + i][p];
    }
  }
  if (tx == 0 && on) {
#pragma unroll
    for (int p = 0; p < PP; ++p) {
      if (j0 + p >= a.k) continue;
      if (a.dw) a.dw[t * a.k + j0 + p] = dot[p];
      if (a.dlogits) {
        if (id[p] < 0 || id[p] >= a.E) flag_status(status, MOE_ERR_INVALID_ARG);
        s_dw[local][j0 + p] = dot[p];
        s_w[local][j0 + p] = w[p];
        s_id[local][j0 + p] = id[p];
      }
    }
  }
  if (!a.dlogits) return;
  __syncthreads();
  if (!on) return;
  float s = 0.f;
  for (int i = 0; i < a.k; ++i) s = fmaf(s_w[local][i], s_dw[local][i], s);
  for (int e = group * nt + tx; e < a.E; e += groups * nt) {
    float g = 0.f;
    for (int i = 0; i < a.k; ++i)
      if (s_id[local][i] == e) g += s_w[local][i] * (s_dw[local][i] - s);
    a.dlogits[t * a.E + e] = g;
  }
}

// Threads per token (a multiple of 32) and tokens per CTA: CTAs of 128 threads, so that fewer wait
// for the slowest of their loads (T = 4096, H = 4096, k = 8: 53.5 us, 56.8 with 256), and of
// 256 with one row per token, whose threads have two loads each (18.0 us, 19.1 with 128).
dim3 rows_block(int nv, int k) {
  const int threads = k == 1 ? kRowsThreads : kRowsThreads / 2;
  int tx = 32;
  while (tx < nv && tx < threads) tx *= 2;
  return dim3(tx, threads / tx);
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
  const dim3 block = rows_block(nv, a.k);
  const dim3 grid((a.T + block.y - 1) / block.y, (nv + block.x - 1) / block.x);
  return launch_kernel(kern, grid, block, 0, st, a, status);
}

#undef MOE_ROWS

cudaError_t launch_unpermute_grad(const UnpermuteGradArgs& a, int sms, int* status, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const int nv = a.H >> 3;
  // warps per pair: more where few pairs would leave the SMs idle
  const int64_t pairs = (int64_t)a.T * a.k;
  int wp = 1;
  while (wp < 4 && wp * 64 < nv && pairs * wp < (int64_t)sms * 16) wp *= 2;
  const bool four = nv <= 64 && a.k > 2 && !a.y_f32 && !a.dout_f32 && pairs >= (int64_t)sms * 16;
  const int groups = four ? (a.k + 3) / 4 : a.k;
  int tokens = 8 / (groups * wp);
  if (tokens < 1) tokens = 1;
  auto kern = a.y_f32      ? (a.dout_f32 ? unpermute_grad_kernel<true, true, 2, 1> : unpermute_grad_kernel<true, false, 2, 1>)
              : a.dout_f32 ? unpermute_grad_kernel<false, true, 2, 1>
              : four       ? unpermute_grad_kernel<false, false, 2, 4>
                           : unpermute_grad_kernel<false, false, 4, 1>;
  return launch_kernel(kern, dim3((a.T + tokens - 1) / tokens), dim3(32 * wp, groups * tokens), 0, st, a, groups,
                       status);
}

}  // namespace moe
