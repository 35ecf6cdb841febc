// moe_combine_norm: the sum of a token's expert rows and what follows the
// block (block_tail.cuh) in one pass over the data.
//
// Each byte of the expert rows, the residual and the outputs moves once, so the
// bound is the copy bandwidth (6770 GB/s measured); sums, norms and scales are
// fp32 and only the stored outputs are rounded.  Device time per call, inputs
// not in L2 (k rows of H per token; "from" are the types of rows and residual):
//   T    H    k                                    us    of the copy bandwidth
//   4096 7168 8  bf16, bf16 -> bf16, x_hat         95    100%
//   4096 4096 8  bf16, bf16 -> bf16, x_hat         57    95%
//   2048 8192 1  bf16, bf16 -> bf16, x_hat         28    71%
//   2048 4096 1  bf16, bf16 -> bf16, x_hat         19    52%
//   2047 5120 1  bf16, fp32 -> fp32, E4M3          24.1  71%
//   333  2944 4  fp32, bf16 -> bf16, E4M3 groups    8.3  37%
//   64   7168 8  bf16, fp32 -> fp32, x_hat          5.5  33%
//   1    4096 8  bf16, bf16 -> bf16, x_hat          3.3  (latency)
// The short calls are a launch, one round of loads and two row reductions.
#include "block_tail.cuh"
#include "kernels.h"
#include "tail.h"
#include "tc_ptx.cuh"

#include <stdlib.h>

#include <atomic>

namespace moe {
namespace {

// ---------------------------------------------------------- per-token parts --
// The tail of one token for a thread that owns VPT 8-column chunks (tid, tid +
// blockDim, ...).  Weights and a per-column gate are read from global memory
// (L1 / L2 resident); the callers supply the sum and the residual.

// Sum (or maximum) over the first nt threads of the CTA (nt a multiple of 32,
// at most 32 NW) with one barrier among them.  `red` (NW floats) must not be
// written again before another such barrier has passed.
template <bool MAX, int NW>
MOE_DEV float rows_reduce(float v, int nt, float (&red)[NW]) {
  v = MAX ? warp_max(v) : warp_sum(v);
  if (nt == 32) return v;
  const int lane = threadIdx.x & 31, nw = nt >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  asm volatile("bar.sync 1, %0;" ::"r"(nt) : "memory");
  v = (lane & (NW - 1)) < nw ? red[lane & (NW - 1)] : 0.f;
#pragma unroll
  for (int o = NW / 2; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  return v;
}

// 1 / norm of the row held in f.
template <int VPT, int NW>
MOE_DEV float row_rnorm(const float (&f)[VPT][8], int nt, int H, float eps, float (&red)[NW]) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) ss = fmaf(f[i][q], f[i][q], ss);
  return 1.0f / sqrtf(rows_reduce<false, NW>(ss, nt, red) / (float)H + eps);
}

// x_hat (and its quantisation) of the row h held in f; chunks beyond the row hold
// zeros.  The norm's weights: KEPT this thread's (one) chunk in `kept`, else the row
// next_w.  red: two arrays of rows_reduce.
template <int VPT, bool KEPT, int NW>
MOE_DEV void write_next(const TailP& p, int t, int H, float (&f)[VPT][8], int nt, const uint4& kept,
                        const bf16* next_w, float (*red)[NW]) {
  const int tid = threadIdx.x, nv = H >> 3;
  const float r = row_rnorm(f, nt, H, p.next_eps, red[0]);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * nt;
    float m = 0.f;
    if (v < nv) {
      float w[8];
      if (KEPT) unpack8_bf16(kept, w);
      else load8(next_w, false, v * 8, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[i][q] = (f[i][q] * r) * w[q];
        m = fmaxf(m, fabsf(f[i][q]));
      }
      if (p.xhat) store8_bf16(p.xhat + (size_t)t * H + v * 8, f[i]);
    }
    amax = fmaxf(amax, m);
    if (p.xq && p.q_group) {
      // a group of 128 columns is 16 consecutive lanes (nt is a multiple of 32,
      // H of 128)
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = tail_scale(m);
      if (v < nv && (v & 15) == 0) p.xscale[(size_t)t * (H >> 7) + (v >> 4)] = s;
      if (v < nv) *reinterpret_cast<uint2*>(p.xq + (size_t)t * H + v * 8) = tail_e4m3x8(f[i], s);
    }
  }
  if (p.xq && !p.q_group) {
    amax = rows_reduce<true, NW>(amax, nt, red[1]);
    const float s = tail_scale(amax);
    if (tid == 0) p.xscale[t] = s;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
      if (v < nv) *reinterpret_cast<uint2*>(p.xq + (size_t)t * H + v * 8) = tail_e4m3x8(f[i], s);
    }
  }
}

// --------------------------------------------------------- one CTA per token --
// Few tokens (latency) and rows too long for the streaming form: every load of
// a chunk (its k expert rows, residual, weights) is issued before the first
// use, so the chain is one round of loads, two row reductions, the stores.
// BJ and EARLY keep the chunks in flight within 128 registers per thread.
struct Raw8 {
  uint4 a, b;  // 8 columns: bf16 in a, or fp32 in a and b
};

MOE_DEV Raw8 ldg8(const void* p, bool f32, size_t at) {
  Raw8 r;
  if (f32) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    r.a = s[0];
    r.b = s[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + at);
    r.b = make_uint4(0u, 0u, 0u, 0u);
  }
  return r;
}

MOE_DEV void raw_to_f(const Raw8& r, bool f32, float (&v)[8]) {
  if (f32) {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
    v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
  } else {
    unpack8_bf16(r.a, v);
  }
}

constexpr int kRowThreads = 512;

template <int VPT, bool YF32>
__global__ void __launch_bounds__(kRowThreads) combine_norm_row_kernel(
    const void* __restrict__ y, int pair_order, const int32_t* __restrict__ row_of_pair, int T, int k,
    int H, const TailP p, int* status) {
  constexpr int BJ = VPT <= 2 ? 8 : 4;  // rows in flight per chunk
  constexpr bool EARLY = VPT <= 2;      // residual held from the start (registers)
  __shared__ float red[3][16];
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x, nv = H >> 3;
  int64_t row[kMaxTopK];  // row of each slot, -1 when skipped
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    row[j] = j < k ? (int64_t)t * k + j : -1;
    if (row_of_pair && j < k) {
      const int r = row_of_pair[row[j]];
      if (r >= T * k && tid == 0) flag_status(status, MOE_ERR_INVALID_ARG);
      if (r < 0 || r >= T * k) row[j] = -1;
      else if (!pair_order) row[j] = r;
    }
  }
  float f[VPT][8];
  Raw8 res[EARLY ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * nt;
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
    if (EARLY) {
      res[i].a = res[i].b = make_uint4(0u, 0u, 0u, 0u);
      if (v < nv && p.residual) res[i] = ldg8(p.residual, p.res_f32 != 0, (size_t)t * H + v * 8);
    }
    if (v >= nv) continue;
#pragma unroll
    for (int j0 = 0; j0 < kMaxTopK; j0 += BJ) {
      Raw8 a[BJ];
#pragma unroll
      for (int j = 0; j < BJ; ++j)
        if (row[j0 + j] >= 0) a[j] = ldg8(y, YF32, (size_t)row[j0 + j] * H + v * 8);
#pragma unroll
      for (int j = 0; j < BJ; ++j) {  // summed in slot order, skipped pairs excluded
        if (row[j0 + j] >= 0) {
          float b[8];
          raw_to_f(a[j], YF32, b);
#pragma unroll
          for (int q = 0; q < 8; ++q) f[i][q] += b[q];
        }
      }
    }
  }
  const int grow = tail_gate_row(p, t, tid == 0 ? status : nullptr);
  const float factor = tail_row_factor(p, grow);
  const float r = p.post_w ? row_rnorm(f, nt, H, p.post_eps, red[0]) : 1.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = tid + i * nt;
    if (v >= nv) continue;
    float h[8], b[8];
    if (EARLY) {
      raw_to_f(res[i], p.res_f32 != 0, b);
    } else if (p.residual) {
      load8(p.residual, p.res_f32 != 0, (size_t)t * H + v * 8, b);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) b[q] = 0.f;
    }
    float w[8] = {};
    if (p.post_w) load8(p.post_w, false, v * 8, w);
    tail_h8(p, H, v * 8, f[i], w, r, grow, factor, b, h);
    store8(p.out, p.out_f32 != 0, (size_t)t * H + v * 8, h);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[i][q] = h[q];
  }
  if (!p.next_w) return;
  write_next<VPT, false>(p, t, H, f, nt, make_uint4(0u, 0u, 0u, 0u), p.next_w, red + 1);
}

// ----------------------------------------------------------- streaming form --
// Persistent CTAs, a token per pass.  The rows a token needs are brought to
// shared memory by bulk copies that a producer warp issues up to S stages
// ahead, so the next rows are in flight while the consumer warps take a token
// through its row reductions.  A stage holds R of the token's k expert rows
// (one copy when they are consecutive); the token's last stage also holds its
// residual and its gate row.  The producer reads the token's indices and
// leaves them beside the rows.  Without the stages the loads of a token wait for
// the reductions of the one before it: 66.7 us instead of 58 at T = 4096, H = 4096,
// k = 8, and 37.1 instead of 24.1 at T = 2047, H = 5120, k = 1.
struct StreamMeta {
  unsigned use;   // slots whose row is present
  float factor;   // tail_row_factor
  int gate_ok;    // 0: gate index out of range
};

constexpr int kWideThreads = 992;  // WIDE: consumers up to this many, else kRowThreads
constexpr int kThreeThreads = 352;  // consumers with VPT = 3 (two CTAs' registers on an SM)

template <int VPT, bool YF32, bool SPLIT, bool WIDE>
__global__ void __launch_bounds__((WIDE ? kWideThreads : (VPT == 3 ? kThreeThreads : kRowThreads)) + 32,
                                  VPT <= 3 && !WIDE ? 2 : 1)
    combine_norm_stream_kernel(const void* __restrict__ y, int pair_order,
                               const int32_t* __restrict__ row_of_pair, int T, int k, int H,
                               const TailP p, int* status, int S, int stage_bytes, int R_,
                               int weights_at) {
  extern __shared__ __align__(128) unsigned char stages[];
  __shared__ uint64_t full[kStreamStages], empty[kStreamStages];
  __shared__ StreamMeta meta[kStreamStages];
  __shared__ float red[2][3][WIDE ? 32 : 16];
  __shared__ int s_abort;
  const int R = SPLIT ? R_ : k;
  const int tid = threadIdx.x, nt = blockDim.x - 32, nv = H >> 3;
  const bool gate_rows = p.gate && p.gate_cols != 1 && !(p.gate_rows == 1 && !p.gate_row);
  const int yb = H * (YF32 ? 4 : 2), rb = p.residual ? H * (p.res_f32 ? 4 : 2) : 0;
  const int gb = gate_rows ? H * (p.gate_f32 ? 4 : 2) : 0;
  pdl_trigger();
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], nt >> 5);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();

  if (tid >= nt) {
    // ------------------------------------------------------------ producer --
    if (tid != nt) return;
    auto copy = [&](unsigned char* dst, const unsigned char* src, int bytes, uint64_t* bar) {
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              ptx::smem_u32(dst)),
          "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
          : "memory");
    };
    const unsigned char* yc = static_cast<const unsigned char*>(y);
    int s = 0, n = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
      int rows[kMaxTopK];
      unsigned use = 0;
      if (row_of_pair) {
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) rows[j] = j < k ? row_of_pair[(int64_t)t * k + j] : -1;
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
          if (rows[j] >= T * k) flag_status(status, MOE_ERR_INVALID_ARG);
          if (rows[j] >= 0 && rows[j] < T * k) use |= 1u << j;
          if (pair_order) rows[j] = t * k + j;
        }
      } else {
        use = (1u << k) - 1;
      }
      const int grow = tail_gate_row(p, t, status);
      const float factor = tail_row_factor(p, grow);
      const bool with_gate = gate_rows && grow >= 0;
      for (int j0 = 0; ok && j0 < k; j0 += R, ++n) {
        if (!(ok = ptx::mbar_wait(&empty[s], ph ^ 1, &s_abort))) break;
        meta[s].use = use;
        meta[s].factor = factor;
        meta[s].gate_ok = grow >= 0;
        unsigned char* st = stages + (size_t)s * stage_bytes;
        const int nr = min(R, k - j0);
        const bool last = j0 + R >= k;
        const unsigned mine = (use >> j0) & ((1u << nr) - 1);
        ptx::mbar_arrive_expect_tx(&full[s], __popc(mine) * yb + (last ? rb + (with_gate ? gb : 0) : 0));
        if (row_of_pair) {
#pragma unroll
          for (int j = 0; j < kMaxTopK; ++j)
            if (j >= j0 && ((mine >> (j - j0)) & 1u))
              copy(st + (size_t)(j - j0) * yb, yc + (size_t)rows[j] * yb, yb, &full[s]);
        } else {
          copy(st, yc + ((size_t)t * k + j0) * yb, nr * yb, &full[s]);
        }
        if (last && rb)
          copy(st + (size_t)R * yb, static_cast<const unsigned char*>(p.residual) + (size_t)t * rb, rb,
               &full[s]);
        if (last && with_gate)
          copy(st + (size_t)R * yb + rb, static_cast<const unsigned char*>(p.gate) + (size_t)grow * gb, gb,
               &full[s]);
        if (++s == S) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok) {
      flag_status(status, MOE_ERR_TIMEOUT);
      // copies in flight must land before the shared memory is given up
      for (int i = n > S ? n - S : 0; i < n; ++i) {
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(&full[i % S], (uint32_t)((i / S) & 1)) &&
               clock64() - t0 < ptx::kSpinLimitCycles) {
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers --
  constexpr int BJ = YF32 ? 2 : 4;
  constexpr bool KEEP = VPT == 1;  // the norm weights stay in registers over the tokens
  uint4 pw = make_uint4(0u, 0u, 0u, 0u), nw = pw;
  if (KEEP && tid < nv) {
    if (p.post_w) pw = reinterpret_cast<const uint4*>(p.post_w)[tid];
    if (p.next_w) nw = reinterpret_cast<const uint4*>(p.next_w)[tid];
  }
  // else in shared memory when the CTA has several tokens (the stages leave little
  // of L1): each thread's own chunks
  const bf16 *post_w = p.post_w, *next_w = p.next_w;
  if (!KEEP && weights_at) {
    uint4* d = reinterpret_cast<uint4*>(stages + weights_at);
    for (int v = tid; p.post_w && v < nv; v += nt) d[v] = reinterpret_cast<const uint4*>(p.post_w)[v];
    if (p.post_w) post_w = reinterpret_cast<const bf16*>(d);
    if (p.post_w) d += nv;
    for (int v = tid; p.next_w && v < nv; v += nt) d[v] = reinterpret_cast<const uint4*>(p.next_w)[v];
    if (p.next_w) next_w = reinterpret_cast<const bf16*>(d);
  }
  int s = 0, n = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int t = blockIdx.x; t < T; t += gridDim.x, ++n) {
    // a wait that runs out leaves garbage in the outputs and is reported
    ok = ptx::mbar_wait(&full[s], ph, &s_abort) && ok;
    const unsigned char* st = stages + (size_t)s * stage_bytes;
    // (a wait that ran out leaves anything here; slots beyond k lie beyond the stage)
    const unsigned use = meta[s].use & ((1u << k) - 1);
    const float factor = meta[s].factor;
    const bool gate_ok = meta[s].gate_ok != 0;
    float f[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int q = 0; q < 8; ++q) f[i][q] = 0.f;
    }
    if (k == 1) {  // one row per token: no loop, no additions
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (use && tid + i * nt < nv) load8(st, YF32, (tid + i * nt) * 8, f[i]);
    } else {
      // summed in slot order, BJ rows' loads at a time; a skipped slot adds 0
#pragma unroll 1
      for (int j0 = 0; SPLIT ? j0 < k : j0 == 0; j0 += R) {
        if (SPLIT && j0 > 0) {  // the stage before this one has been read
          __syncwarp();
          if ((tid & 31) == 0) ptx::mbar_arrive(&empty[s]);
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
          ok = ptx::mbar_wait(&full[s], ph, &s_abort) && ok;
          st = stages + (size_t)s * stage_bytes;
        }
        const unsigned mine = SPLIT ? (use >> j0) & ((1u << R) - 1) : use;
        const int nr = SPLIT ? min(R, k - j0) : k;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = tid + i * nt;
          if (v >= nv) continue;
#pragma unroll 1
          for (int j1 = 0; j1 < nr; j1 += BJ) {
            Raw8 a[BJ];
#pragma unroll
            for (int j = 0; j < BJ; ++j) {
              a[j].a = a[j].b = make_uint4(0u, 0u, 0u, 0u);
              if ((mine >> (j1 + j)) & 1u) a[j] = ldg8(st + (size_t)(j1 + j) * yb, YF32, v * 8);
            }
#pragma unroll
            for (int j = 0; j < BJ; ++j) {
              float b[8];
              raw_to_f(a[j], YF32, b);
#pragma unroll
              for (int q = 0; q < 8; ++q) f[i][q] += b[q];
            }
          }
        }
      }
    }
    const float r = p.post_w ? row_rnorm(f, nt, H, p.post_eps, red[n & 1][0]) : 1.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = tid + i * nt;
      if (v >= nv) continue;
      float a[8];
      if (p.post_w) {
        if (KEEP) unpack8_bf16(pw, a);
        else load8(post_w, false, v * 8, a);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[i][q] = (f[i][q] * r) * a[q];
      }
      if (p.gate && p.gate_cols != 1 && gate_ok) {
        if (gate_rows) load8(st + (size_t)R * yb + rb, p.gate_f32 != 0, v * 8, a);
        else load8(p.gate, p.gate_f32 != 0, v * 8, a);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[i][q] *= a[q];
      }
      float h[8];
      if (rb) {
        load8(st + (size_t)R * yb, p.res_f32 != 0, v * 8, h);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) h[q] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (gate_ok) h[q] = fmaf(factor, f[i][q], h[q]);
        f[i][q] = h[q];
      }
      store8(p.out, p.out_f32 != 0, (size_t)t * H + v * 8, h);
    }
    // this warp has read the stage
    __syncwarp();
    if ((tid & 31) == 0) ptx::mbar_arrive(&empty[s]);
    if (p.next_w)
      write_next<VPT, KEEP>(p, t, H, f, nt, nw, next_w, red[n & 1] + 1);
    if (++s == S) {
      s = 0;
      ph ^= 1;
    }
  }
  if (!ok) flag_status(status, MOE_ERR_TIMEOUT);
}

template <int VPT, bool YF32>
cudaError_t launch_row(const void* y, bool pair_order, const int32_t* row_of_pair, int T, int k, int H,
                       const TailP& p, int* status, int threads, cudaStream_t st) {
  return launch_kernel(combine_norm_row_kernel<VPT, YF32>, dim3(T), dim3(threads), 0, st, y,
                       (int)pair_order, row_of_pair, T, k, H, p, status);
}

// cudaErrorNotSupported when even one expert row per stage does not fit twice;
// with `two` also unless two CTAs of two whole tokens each fit an SM (or every token
// gets a CTA at once).
template <int VPT, bool YF32, bool WIDE>
cudaError_t launch_stream(const void* y, bool pair_order, const int32_t* row_of_pair, int T, int k, int H,
                          const TailP& p, int* status, int sms, int threads, bool two, cudaStream_t st) {
  auto kern = combine_norm_stream_kernel<VPT, YF32, false, WIDE>;
  static std::atomic<int> regs{0};  // of the kernel's threads
  cudaError_t e = cudaSuccess;
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  const int64_t yb = (int64_t)H * (YF32 ? 4 : 2);
  const int64_t extra = (p.residual ? (int64_t)H * (p.res_f32 ? 4 : 2) : 0) +
                        (p.gate && p.gate_cols != 1 ? (int64_t)H * (p.gate_f32 ? 4 : 2) : 0);
  auto bytes = [&](int rows) { return (rows * yb + extra + 127) / 128 * 128; };
  // CTAs an SM holds by registers (given out to four warps at a time) and threads
  const int warps = (threads / 32 + 1 + 3) / 4 * 4;
  int by_regs = 65536 / ((regs.load(std::memory_order_relaxed) + 7) / 8 * 8 * 32 * warps);
  if (by_regs > 2048 / (threads + 32)) by_regs = 2048 / (threads + 32);
  if (by_regs > kStreamCtas) by_regs = kStreamCtas;
  if (by_regs < 1) return cudaErrorNotSupported;
  int64_t weights = 0;  // of the norms, in shared memory
  auto by_smem = [&](int64_t b) { return (int)(kStreamSmem / (b + kStreamStatic + weights)); };
  int R = k, S, per_sm = by_smem(bytes(k)) < by_regs ? by_smem(bytes(k)) : by_regs;
  if (per_sm > 0 && T <= sms * per_sm) {
    // every token gets a CTA of its own at once: one stage each.  Against two stages and
    // fewer CTAs: T = 450, H = 5120, k = 1 4.85 us, 5.19; T = 200, H = 4096, k = 8 5.46, 5.43;
    // T = 333, H = 2944, k = 4 8.3 either way; with short rows it loses (T = 400, H = 1024,
    // k = 8 4.17, 3.41)
    S = 1;
  } else {
    // two or more stages, each as much of a token as fits (a whole token wherever two
    // fit: copies stay long, and a token waits once); then as many CTAs as fit, then
    // the memory that is left goes to more stages
    auto plan = [&](int& rows, int& ctas) {
      rows = k;
      while (rows > 1 && by_smem(2 * bytes(rows)) < 1) rows = (rows + 1) / 2;
      ctas = by_smem(2 * bytes(rows)) < by_regs ? by_smem(2 * bytes(rows)) : by_regs;
    };
    plan(R, per_sm);
    if (per_sm < 1 || (two && (R < k || per_sm < 2))) return cudaErrorNotSupported;
    if (VPT > 1) {
      // the norms' weights beside the stages (H = 12288, k = 1: 40.1 us, 54.5 without;
      // H = 8192, k = 6: 109, 121 without), unless that leaves stages of one row (H = 15872,
      // k = 8: 185, 132 without) or fewer CTAs: one instead of two (H = 7168, k = 1, fp32
      // residual, T = 2048: 43.5, 37.4 without), or with more than one row per token two
      // instead of three (H = 5120: k = 2 47.2, 44.0 without; but k = 1 34.7, 37.9 without)
      int rows, ctas;
      weights = (int64_t)H * ((p.post_w ? 2 : 0) + (p.next_w ? 2 : 0));
      plan(rows, ctas);
      if (ctas < 1 || (rows == 1 && R > 1) || (ctas < per_sm && (k > 1 || ctas < 2))) {
        weights = 0;
      } else {
        R = rows;
        per_sm = ctas;
      }
    }
    S = (int)((kStreamSmem / per_sm - kStreamStatic - weights) / bytes(R));
    if (S > kStreamStages) S = kStreamStages;
    // (part of a token per stage: never with VPT = 3, which takes whole tokens only, and never
    // with bf16 rows of up to 512 chunks, of which two whole tokens always fit: at most 96 KB
    // each with eight rows, an fp32 residual and an fp32 gate row)
    if constexpr (VPT == 2 || VPT == 4 || (VPT == 1 && (YF32 || WIDE))) {
      if (R < k) kern = combine_norm_stream_kernel<VPT, YF32, true, WIDE>;
    } else if (R < k) {
      return cudaErrorNotSupported;
    }
  }
  const size_t smem = (size_t)S * bytes(R) + weights;
  // the same limit in every call: another thread's launch may lie between this and ours
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem - kStreamStatic);
  if (e != cudaSuccess) return e;
  const int grid = T < sms * per_sm ? T : sms * per_sm;
  return launch_kernel(kern, dim3(grid), dim3(threads + 32), smem, st, y, (int)pair_order, row_of_pair, T,
                       k, H, p, status, S, (int)bytes(R), R, weights ? (int)(S * bytes(R)) : 0);
}

}  // namespace

cudaError_t launch_combine_norm(const void* y, bool y_f32, bool pair_order,
                                const int32_t* row_of_pair, int T, int k, int H, const TailP& p,
                                int* status, int sms, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const int nv = H / 8;
  // A CTA per token while the SMs hold all tokens at once, the streaming form beyond:
  // T = 64 (H = 7168, k = 8) 5.5 us against 6.0 streamed; T = 333 (H = 2944, k = 4)
  // 10.6 against 8.3.  Rows above 16384 columns always take a CTA per token: a thread
  // of the streaming form would hold more than four chunks.  MOE_CN_STREAM=0|1 sets the
  // form for measurements.
  const char* env = getenv("MOE_CN_STREAM");
  if (nv <= 2048 && (env ? env[0] == '1' : T > sms)) {
    // Consumers and chunks per consumer (T = 2048, bf16, in us).  Where a token has few bytes of
    // expert rows, its two reductions are most of a CTA's time, and two or three CTAs
    // on an SM overlap them: the fewest chunks with which two fit (k = 1: H = 4096 19.0 with
    // two chunks, 23.3 with one and a single CTA; H = 5120 21.3, 24.6 by 640 threads; H = 8192
    // 28.2 with three, 37.2 with two).  With more rows the instructions and shared
    // loads of the sums count, and more warps overlap those: H = 7168, k = 4 35.4 with 896
    // threads, 43.2 with 448 of two chunks; k = 8 51.1, 61.2; H = 4096, k = 8 31.3 with one
    // chunk, 40.7 with two; H = 12288 103 with two, 123 with four.  The border is at 4
    // bytes per column (fp32, H = 5120, k = 2: 29.5 against 35.5), and at 8 for rows of up to 512
    // chunks, whose one CTA has only 512 threads (k = 4, H = 4096: 24.6 against 26.4; not for up
    // to two tokens per SM: T = 200 5.8 against 4.8).
    cudaError_t e = cudaErrorNotSupported;
#define MOE_CN(V, W, TWO)                                                                             \
  {                                                                                                   \
    const int threads = ((nv + V - 1) / V + 31) / 32 * 32;                                            \
    e = y_f32 ? launch_stream<V, true, W>(y, pair_order, row_of_pair, T, k, H, p, status, sms,        \
                                          threads, TWO, st)                                           \
              : launch_stream<V, false, W>(y, pair_order, row_of_pair, T, k, H, p, status, sms,       \
                                           threads, TWO, st);                                         \
  }
    const int row_bytes = k * (y_f32 ? 4 : 2);  // per column
    if (nv <= kRowThreads ? row_bytes <= 8 && T > 2 * sms : row_bytes <= 4) {
      if (nv <= kRowThreads) MOE_CN(1, false, true)
      if (e == cudaErrorNotSupported && nv <= 2 * kRowThreads) MOE_CN(2, false, true)
      if (e == cudaErrorNotSupported && nv > kWideThreads && nv <= 3 * kThreeThreads) MOE_CN(3, false, true)
    }
    if (e == cudaErrorNotSupported) {
      if (nv <= kRowThreads) MOE_CN(1, false, false)
      else if (nv <= kWideThreads) MOE_CN(1, true, false)
      else if (nv <= 2 * kRowThreads) MOE_CN(2, false, false)
      else if (nv <= 2 * kWideThreads) MOE_CN(2, true, false)
      else MOE_CN(4, false, false)
    }
#undef MOE_CN
    if (e != cudaErrorNotSupported) return e;
  }
  const int vpt = nv <= 512 ? 1 : (nv <= 1024 ? 2 : (nv <= 2048 ? 4 : 8));
  const int threads = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
#define MOE_CN(V)                                                                                     \
  return y_f32 ? launch_row<V, true>(y, pair_order, row_of_pair, T, k, H, p, status, threads, st)     \
               : launch_row<V, false>(y, pair_order, row_of_pair, T, k, H, p, status, threads, st)
  if (vpt == 1) MOE_CN(1);
  if (vpt == 2) MOE_CN(2);
  if (vpt == 4) MOE_CN(4);
  MOE_CN(8);
#undef MOE_CN
}

}  // namespace moe
