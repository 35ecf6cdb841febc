// Dense product with bias, activation and residual in its epilogue
// (moe_linear), and the products of its gradient (moe_linear_backward):
//   out  = residual + act(x W^T + b)
//   dpre = dout act'(pre),  dx = dpre W,  dW = dpre^T x,  db = sum_m dpre
//
// All three products are D[q, p] = sum_k a[p, k] b[q, k] with p the contiguous
// index of the output and each operand K-major ([rows, K] in memory) or MN-major
// ([K, rows]):
//   forward  a = W  [N, K]         b = x [M, K]
//   dx       a = W  stored [K, P]  b = dpre [M, N]
//   dW       a = x  stored [K, P]  b = dpre stored [K, Q]
// The tensor cores take both layouts from shared memory (tcgen05 descriptors), so
// nothing is transposed.  Three forms, chosen in launch_product by their measured times: a
// kernel for one token, clusters that split K, and pairs of CTAs.  Device time per call,
// inputs not in L2, against bytes at 6794 GB/s or FLOPs at 1952 TFLOP/s:
//   M x N x K                 us      of the floor
//   8192 x 8192 x 8192        539-582 0.97-1.05  pairs (under the power limit)
//   4096 x 12288 x 4096       216-224 0.94-0.98  pairs; GELU and kept values 238, 0.89, with the
//                                            tanh form 227-234, 0.90-0.93 (257, 0.82, back to back
//                                            under the power limit); fp32 output 243-251
//     dx, dW of it            233, 216  0.90, 0.97
//     its gradient, SiLU, db  492-512   0.83-0.86  (550, 0.77, back to back); fp32 dout and dW 545
//     16, 64, 256 rows of 4096 x 4096   31, 33, 38 us, 0.3: four launches
//   1024 x 4096 x 4096        25      0.70   pairs, one round of 64 of 76
//   256 x 4096 x 4096         15.8    0.35   split, 128 CTAs
//   512 x 1024 x 1024         7.4     0.08   split, 64 columns, four CTAs a tile
//   61 x 7168 x 2048          10.7    0.43   split
//   16 x 4096 x 4096          10.3    0.48   split
//   1 x 12288 x 4096          17.7-18.6  0.80-0.84   one token
//   1 x 4096 x 4096           7.3     0.67   one token
// Small ones are a launch (1.7 us for one token, 3.4 with TMEM and a cluster), the ramp of the
// loads and the reduction over the cluster; large ones the tensor pipe.
#include <cuda.h>
#include <string.h>

#include "block_tail.cuh"
#include "column_sum.cuh"
#include "common.cuh"
#include "device_counts.h"
#include "tc_common.cuh"
#include "tc_ptx.cuh"
#include "train.h"

namespace moe {
namespace {

using namespace ptx;
using namespace tc;

constexpr int kTileP = 128;    // rows of a per CTA (MMA M)
constexpr int kStepK = 64;     // K of a ring stage: 128 bytes
constexpr int kMaxRing = 12;
constexpr int kBoxBytes = 64 * 128;  // an MN-major box: 64 K rows of 64 elements
constexpr int kLinThreads = 320;     // producer, MMA issuer, eight epilogue warps
constexpr int kEpiWarps = 8;
// The tensor cores' fp32 additions truncate.  Over n terms of mixed signs that leaves about 1.1e-9 n
// of the sum (measured: 9e-7 at n = 1024, 1.9e-5 at 16384), over terms of one sign, where
// it adds up, 1.7e-9 n to 6e-9 n (1.3e-6 at 768, 8e-5 at 16384, 1.6e-3 at 262144).
// fp32 results: sums longer than kSegSteps stages go through registers, rounded to nearest,
// every kSegSteps stages, which leaves about 7e-7, 1.3e-6 with one sign (16 stages 1e-6, 8 stages
// 5e-7; 4096 x 12288 x 4096 249 us, 238 and 263).
// bf16 results: half a step is 2^-8 of the value.  What a CTA adds up over kLongSteps stages (16384
// terms) is off by a fiftieth of that at most and is taken whole; longer sums go through
// registers every kLongSeg stages.
constexpr int kSegSteps = 12;
constexpr int kLongSteps = 256;
constexpr int kLongSeg = 64;

// ------------------------------------------------------------- activations --
// The epilogues run under the next tile's products, and with short K they are what
// takes the time, so each activation is a few products around one 2^x and one reciprocal
// (both within two units in the last place; results below 2^-126 are 0).
MOE_DEV float exp2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
MOE_DEV float recip_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + 2^u); 0 where 2^u is infinite.
MOE_DEV float sigmoid2_f(float u) { return recip_f(1.0f + exp2_f(u)); }

// 0.5 (1 + tanh(a (z + b z^3))) = sigmoid(2 a (z + b z^3)): no difference of near values.
MOE_DEV float gelu_tanh_gate(float z) {
  return sigmoid2_f(z * fmaf(z * z, -2.0f * kGeluA * kGeluB * kLog2E, -2.0f * kGeluA * kLog2E));
}

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).
// Phi(-|z|) = e t (p0 + ... + p7 t^7), t = 1 / (1 + 0.3 |z|): the polynomial is a fit to
// exp(z^2 / 2) Phi(-|z|) / t on 0 <= |z| <= 13.4 by least squares, weighted until the
// largest relative error was least, 1.3e-7; past that e is 0.  So the lower tail keeps its
// relative precision but for the rounding of z^2, as exp does.
MOE_DEV float normal_cdf(float z, float& e) {
  const float t = recip_f(fmaf(fabsf(z), 0.3f, 1.0f));
  e = exp2_f(z * z * (-0.5f * kLog2E));
  float p = fmaf(t, 0.035966480f, -0.158421054f);
  p = fmaf(t, p, 0.208457217f);
  p = fmaf(t, p, -0.055625346f);
  p = fmaf(t, p, 0.129592260f);
  p = fmaf(t, p, 0.099599972f);
  p = fmaf(t, p, 0.120804417f);
  p = fmaf(t, p, 0.119625991f);
  const float q = t * p * e;
  return z > 0.f ? 1.0f - q : q;
}

MOE_DEV float act_f(float z, int act) {
  float e;
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActSilu: return z * sigmoid2_f(z * -kLog2E);
    case kActGelu: return z * normal_cdf(z, e);
    case kActGeluTanh: return z * gelu_tanh_gate(z);
    default: return z;
  }
}

// The choice once for N values.
template <int N>
MOE_DEV void act_all(float* v, int act) {
#define MOE_ACT(A)                                       \
  case A:                                                \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = act_f(v[i], A); \
    break;
  switch (act) {
    MOE_ACT(kActRelu)
    MOE_ACT(kActSilu)
    MOE_ACT(kActGelu)
    MOE_ACT(kActGeluTanh)
    default: break;
  }
#undef MOE_ACT
}

MOE_DEV float act_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActSilu: {
      const float p = sigmoid2_f(z * -kLog2E);
      return p * fmaf(z, 1.0f - p, 1.0f);
    }
    case kActGelu: {
      float e;
      const float c = normal_cdf(z, e);
      return e == 0.f ? c : fmaf(z * 0.3989422804014327f, e, c);
    }
    case kActGeluTanh: {
      const float s = gelu_tanh_gate(z);
      const float t = s * (1.0f - s);  // 0 where z^3 is past the exponent's range
      return t == 0.f ? s : fmaf(z * t, 2.0f * kGeluA * fmaf(z * z, 3.0f * kGeluB, 1.0f), s);
    }
    default: return 1.f;
  }
}

// ------------------------------------------------------------- the epilogue --
struct Epi {
  const void* bias;
  const void* residual;
  bf16* pre;
  void* out;
  int act;
  int bias_f32, res_f32, out_f32;
  int64_t P, Q;
};

// Four columns p .. p + 3 of row q.
MOE_DEV void epilogue4(const Epi& e, int64_t q, int64_t p, float (&v)[4]) {
  const int64_t at = q * e.P + p;
  if (e.bias) {
    if (e.bias_f32) {
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(e.bias) + p);
      v[0] += b.x; v[1] += b.y; v[2] += b.z; v[3] += b.w;
    } else {
      const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(e.bias) + p);
      v[0] += bf16_lo(b.x); v[1] += bf16_hi(b.x); v[2] += bf16_lo(b.y); v[3] += bf16_hi(b.y);
    }
  }
  if (e.pre)
    *reinterpret_cast<uint2*>(e.pre + at) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
  act_all<4>(v, e.act);
  if (e.residual) {
    if (e.res_f32) {
      const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + at);
      v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(e.residual) + at);
      v[0] += bf16_lo(r.x); v[1] += bf16_hi(r.x); v[2] += bf16_lo(r.y); v[3] += bf16_hi(r.y);
    }
  }
  if (e.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(e.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<bf16*>(e.out) + at) =
        make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
}

// The warp's wait: false in all lanes if it ran out in one of them.  What follows a wait (elect.sync, tcgen05
// instructions, __syncwarp) needs the whole warp, without a limit, and a lane that left its role alone
// would never reach it.  (The vote is also what a stage's lanes meet at: with a __syncwarp beside it
// large products take 1.5% longer; one thread per role instead of a warp, 30%.)
MOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// ------------------------------------------------------- cluster split-K form --
// A tile is 128 columns p x BN rows q; the CTAs of a cluster take consecutive parts
// of K.  Each leaves its fp32 tile in its shared memory (over the ring), then
// every CTA adds a share of the tile's elements over the cluster in rank order and
// runs the epilogue on them: no workspace, no atomics, the same bits every time.
// Few tiles with a long K are what bounds it: so the tile's width is chosen with S (below).
constexpr int kMaxSplit = 16;  // CTAs of a cluster: 1 to 8, or 16

struct SplitP {
  Epi e;
  int steps;        // stages of the whole K
  int ring, stage_bytes;
  int seg;          // stages added up in the tensor cores
  int* status;
};

// Units (four columns of a row) u0 .. u1 - 1 of the tile, added over the S CTAs in rank order.
// (256 x 4096 x 64, no split: 7.6 us, 11.6 with S as a variable and predicated steps up to eight;
// 256 x 4096 x 4096, four CTAs: 15.7 us, 19.6 with 32 bytes per lane and load.)
template <int S>
MOE_DEV void split_store(const Epi& e, uint32_t base, int u0, int u1, int64_t p0, int64_t q0) {
  uint32_t at[S];
#pragma unroll
  for (int r = 0; r < S; ++r) at[r] = S == 1 ? base : cluster_addr(base, r);
#pragma unroll S > 8 ? 1 : 2
  for (int u = u0 + threadIdx.x; u < u1; u += kLinThreads) {
    const int64_t pc = p0 + (u & 31) * 4;
    if (pc >= e.P) continue;
    float4 w[S];
#pragma unroll
    for (int r = 0; r < S; ++r) w[r] = S == 1 ? shared_ld4(at[r] + u * 16) : cluster_ld4(at[r] + u * 16);
    float v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int r = 1; r < S; ++r) {
      v[0] += w[r].x; v[1] += w[r].y; v[2] += w[r].z; v[3] += w[r].w;
    }
    epilogue4(e, q0 + (u >> 5), pc, v);
  }
}

template <bool A_MN, bool B_MN, int BN>
__global__ void __launch_bounds__(kLinThreads, BN <= 64 ? 2 : 1)
    product_split_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                         const SplitP p) {
  constexpr int HC = BN >= 32 ? BN / 2 : 16;           // columns of an epilogue warp
  constexpr int ACC = BN < 32 ? 32 : BN;               // TMEM columns of a buffer
  constexpr int TMEM = 2 * ACC < 32 ? 32 : 2 * ACC;
  constexpr int kBBoxes = B_MN ? (BN + 63) / 64 : 1;
  extern __shared__ unsigned char dyn[];
  __shared__ uint64_t full[kMaxRing], empty[kMaxRing], tfull[2], tempty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  unsigned char* ring = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x, S = gridDim.x;  // the cluster is the grid's x
  const int64_t p0 = (int64_t)blockIdx.y * kTileP, q0 = (int64_t)blockIdx.z * BN;
  const int k0 = (int)((int64_t)p.steps * rank / S), k1 = (int)((int64_t)p.steps * (rank + 1) / S);

  if (warp == 0 && lane == 0) {
    s_abort = 0;
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_mbar_init();
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
  } else if (warp == 1) {
    tmem_alloc(&s_tmem, TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // (not before the allocation: the next kernel's waits for this one's)
  pdl_wait();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    // -------------------------------------------------------------- producer --
    int s = 0;
    uint32_t ph = 0, armed = 0, armed_ph = 0;
    bool ok = true;
    for (int k = k0; k < k1; ++k) {
      if (!(ok = warp_wait(&empty[s], ph ^ 1, &s_abort))) break;
      if (elect_one()) {
        unsigned char* a = ring + (size_t)s * p.stage_bytes;
        unsigned char* b = a + kTileP * 128;
        mbar_arrive_expect_tx(&full[s], kTileP * 128 + (B_MN ? kBBoxes * kBoxBytes : BN * 128));
        if (A_MN) {
          for (int i = 0; i < 2; ++i) tma_load_2d_plain(a + i * kBoxBytes, &ta, &full[s], (int)p0 + 64 * i, k * kStepK);
        } else {
          tma_load_2d_plain(a, &ta, &full[s], k * kStepK, (int)p0);
        }
        if (B_MN) {
          for (int i = 0; i < kBBoxes; ++i)
            tma_load_2d_plain(b + i * kBoxBytes, &tb, &full[s], (int)q0 + 64 * i, k * kStepK);
        } else {
          tma_load_2d_plain(b, &tb, &full[s], k * kStepK, (int)q0);
        }
      }
      armed |= 1u << s;
      armed_ph = (armed_ph & ~(1u << s)) | (ph << s);
      if (++s == p.ring) {
        s = 0;
        ph ^= 1;
      }
    }
    if (ok) ok = __all_sync(0xffffffffu, producer_tail(empty, p.ring, s, ph, &s_abort));
    if (!ok) {
      if (lane == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
      drain_armed(full, p.ring, armed, armed_ph);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer --
    const uint32_t idesc = make_idesc_major(kTileP, BN, A_MN, B_MN);
    int s = 0, buf = 0, n = 0;
    uint32_t ph = 0, bph = 0;
    bool ok = true, issued = false;
    for (int k = k0; k < k1; ++k) {
      if (n == 0) {
        if (!(ok = warp_wait(&tempty[buf], bph ^ 1, &s_abort))) break;
        tc_fence_after();
      }
      if (!(ok = warp_wait(&full[s], ph, &s_abort))) break;
      tc_fence_after();
      const uint32_t a = smem_u32(ring + (size_t)s * p.stage_bytes), b = a + kTileP * 128;
      const bool last = k + 1 == k1 || n + 1 == p.seg;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ad = A_MN ? sw128_mn_desc(a + kk * 2048, 64) : sw128_desc(a + kk * 32);
          const uint64_t bd = B_MN ? sw128_mn_desc(b + kk * 2048, 64) : sw128_desc(b + kk * 32);
          mma_bf16(tmem + buf * ACC, ad, bd, idesc, (n | kk) ? 1u : 0u);
        }
        mma_commit(&empty[s]);
        if (last) mma_commit(&tfull[buf]);
      }
      issued = true;
      if (++s == p.ring) {
        s = 0;
        ph ^= 1;
      }
      ++n;
      if (last) {
        n = 0;
        if (++buf == 2) {
          buf = 0;
          bph ^= 1;
        }
      }
    }
    if (ok) ok = __all_sync(0xffffffffu, accumulator_tail(tempty, buf, bph, &s_abort));
    if (!ok) {
      if (lane == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
      if (issued) {  // issued MMAs complete before TMEM is released
        if (elect_one()) mma_commit(&drain);
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try_wait(&drain, 0) && clock64() - t0 < kSpinLimitCycles) {
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue --
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const bool mine = BN >= 32 || half == 0;
    float acc[HC];
    int buf = 0;
    uint32_t bph = 0;
    bool ok = true;
    for (int k = k0; k < k1; k += p.seg) {
      if (!(ok = warp_wait(&tfull[buf], bph, &s_abort))) break;
      tc_fence_after();
      if (mine) {
        const uint32_t at = tmem + buf * ACC + half * HC + ((uint32_t)(quarter * 32) << 16);
        if (k == k0) {
          if constexpr (HC <= 16) tmem_ld16(at, acc);
          else {
#pragma unroll
            for (int i = 0; i < HC; i += 32) tmem_ld32(at + i, acc + i);
          }
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < HC; i += 16) {
            float v[16];
            tmem_ld16(at + i, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i + j] += v[j];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
      if (++buf == 2) {
        buf = 0;
        bph ^= 1;
      }
    }
    if (!ok && lane == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
    // (the last tfull says that every MMA has read its stage: the ring is free)
    if (ok && mine) {
      float* t = reinterpret_cast<float*>(ring) + (size_t)(half * HC) * kTileP + quarter * 32 + lane;
#pragma unroll
      for (int i = 0; i < HC; ++i) t[i * kTileP] = acc[i];
    }
  }
  __syncwarp();
  cluster_sync();
  {
    const int rows = (int)(p.e.Q - q0 < BN ? p.e.Q - q0 : BN);
    const int units = rows * (kTileP / 4);
    const int u0 = (int)((int64_t)units * rank / S), u1 = (int)((int64_t)units * (rank + 1) / S);
    const uint32_t base = smem_u32(ring);
#define MOE_S(N) \
  case N: split_store<N>(p.e, base, u0, u1, p0, q0); break
    switch (S) {
      MOE_S(1); MOE_S(2); MOE_S(3); MOE_S(4); MOE_S(5); MOE_S(6); MOE_S(7); MOE_S(8); MOE_S(16);
    }
#undef MOE_S
  }
  cluster_sync();  // the others have read this CTA's tile
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM);
}

// --------------------------------------------------------------- one token --
// One row of b, both operands K-major: no tensor cores.  Each warp streams kRowsR rows
// of a (weights) once, 16 bytes per lane and load, kRowsUnroll loads of each in flight,
// against b's row from L1; W warps share a row's K where there are few rows.
// Products are exact in fp32 and added with fma.  The bound is the copy bandwidth and
// a launch: there are no barriers, TMEM or clusters to set up.  4096 x 4096 7.0 us (the
// cluster form 9.4; two tokens 9.7 in the cluster form, 10.3 so), 12288 x 4096 17.7 (20.0);
// 4 rows x 2 loads against 2 x 4: 7.0, 8.7; weights kept out of L1: 7.9, 8.4 before.
constexpr int kRowsWarps = 4;
constexpr int kRowsUnroll = 2;
constexpr int kRowsR = 4;

MOE_DEV void unpack_pairs(const uint4& u, float2 (&f)[4]) {
  f[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x));
  f[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
  f[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z));
  f[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
}

// 16 bytes that are read once: not kept in L1, where b's rows are.
MOE_DEV uint4 load_once(const bf16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(kRowsWarps * 32) product_token_kernel(const bf16* __restrict__ a,
                                                                        const bf16* __restrict__ b, int64_t K, int W,
                                                                        const Epi e) {
  constexpr int R = kRowsR;
  __shared__ float red[kRowsWarps][R];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % W, group = warp / W;
  const int64_t p0 = ((int64_t)blockIdx.x * (kRowsWarps / W) + group) * R;
  const int nk = (int)(K >> 3), step = 32 * W;
  float2 acc[R] = {};
  for (int k0 = sub * 32 + lane; k0 < nk; k0 += step * kRowsUnroll) {
    uint4 w[kRowsUnroll][R];
#pragma unroll
    for (int i = 0; i < kRowsUnroll; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        w[i][r] = make_uint4(0u, 0u, 0u, 0u);
        if (k0 + i * step < nk && p0 + r < e.P) w[i][r] = load_once(a + (p0 + r) * K + (int64_t)(k0 + i * step) * 8);
      }
#pragma unroll
    for (int i = 0; i < kRowsUnroll; ++i) {
      if (k0 + i * step >= nk) break;
      float2 x[4];
      unpack_pairs(*reinterpret_cast<const uint4*>(b + (int64_t)(k0 + i * step) * 8), x);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 f[4];
        unpack_pairs(w[i][r], f);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[r] = fma_f2(f[q], x[q], acc[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float v = warp_sum(acc[r].x + acc[r].y);
    if (lane == 0) red[warp][r] = v;
  }
  if (W > 1) __syncthreads();
  else __syncwarp();
  const int64_t p = p0 + lane;
  if (sub != 0 || lane >= R || p >= e.P) return;
  float v = 0.f;
  for (int i = 0; i < W; ++i) v += red[warp + i][lane];
  auto get = [](const void* s, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(s)[i] : __bfloat162float(static_cast<const bf16*>(s)[i]);
  };
  if (e.bias) v += get(e.bias, e.bias_f32, p);
  if (e.pre) e.pre[p] = __float2bfloat16_rn(v);
  act_all<1>(&v, e.act);
  if (e.residual) v += get(e.residual, e.res_f32, p);
  if (e.out_f32) static_cast<float*>(e.out)[p] = v;
  else static_cast<bf16*>(e.out)[p] = __float2bfloat16_rn(v);
}

// -------------------------------------------------------------- CTA-pair form --
// Persistent pairs of CTAs (cluster of two), a tile of 256 rows q x BN columns p
// at a time: each CTA of a pair loads its 128 rows and half of the columns, and the
// MMAs of the pair, issued by its first CTA, take both halves (tcgen05
// cta_group::2): 32 KB per 128 x 256 x 64 products of a CTA instead of the 48 KB of
// a single one.  Two accumulators in TMEM, so that the eight epilogue warps of a
// tile run under the products of the next.
struct PairP {
  Epi e;
  int steps, ring, stage_bytes;
  int tq, tp;       // tiles of 256 x 256 along q and p
  int whole;        // tiles taken whole; those after them in two halves of 128 columns
  int group;        // row tiles of a raster group
  int seg;          // KEEP: stages added up in the tensor cores at a time
  int* status;
};

// Unit u: rows q .. q + 255, columns c .. c + 2 half - 1.  Tiles in groups of `group`
// row tiles, rows fastest within a group: the tiles in flight share their operands in
// L2.  A tile with no more than 128 columns left in the matrix has them alone; the
// second half of such a tile is no work (half 0).
MOE_DEV void pair_unit(const PairP& p, int u, int& q, int& c, int& half) {
  const bool split = u >= p.whole;
  const int t = split ? p.whole + ((u - p.whole) >> 1) : u;
  const int per = p.group * p.tp, g = t / per, r = t - g * per;
  const int rows = min(p.group, p.tq - g * p.group);
  c = r / rows;
  q = (g * p.group + (r - c * rows)) * 256;
  c *= 256;
  half = 128;
  if (split || p.e.P - c <= 128) half = 64;
  if (split && ((u - p.whole) & 1)) {
    c += 128;
    if (c >= p.e.P) half = 0;
  }
}

// A warp's 32 rows x W words (128 bytes; 32 of bf16 results beside 128 kept sums, which leave few
// registers: 128 bytes of them spill so, 356 with 64-byte rows) on their way out: each lane
// writes its row's words in 16-byte chunks at the places of the 128-byte (32-byte) swizzle, and one lane hands them to a TMA store, which writes whole lines and drops
// what lies outside the matrix.
// (Straight from registers, 32 bytes of 32 rows at a time: 38.6 us instead of 29.7
// at 4096 x 12288 x 64.)
constexpr int kStoreBytes = 32 * 128;

// Columns of a store.
constexpr int pair_box(bool f32, bool keep) { return f32 ? 32 : (keep ? 16 : 64); }

template <int W>
MOE_DEV void store_box(unsigned char* stage, int lane, const uint32_t (&w)[W], const CUtensorMap* map, int x,
                       int y) {
  static_assert(W == 32 || W == 8, "a row of 128 or 32 bytes");
  const int swizzle = W == 32 ? lane & 7 : (lane >> 2) & 1;
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int j = 0; j < W / 4; ++j)
    *reinterpret_cast<uint4*>(stage + lane * (4 * W) + ((j ^ swizzle) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, stage, x, y);
    bulk_commit();
  }
}

// Columns p .. p + N - 1 of the warp's 32 rows,
// one row per lane (q: this lane's, q0: the first); the first column is below P, a
// multiple of 8.  Rows from Q on hold values of no row and are dropped.
template <bool F32, int N>
MOE_DEV void epilogue_box(const Epi& e, int64_t q, int64_t q0, int64_t p, float* v, unsigned char* stage, int lane,
                          const CUtensorMap* tout, const CUtensorMap* tpre) {
  constexpr int W = F32 ? N : N / 2;
  const int groups = (int)min((int64_t)(N / 8), (e.P - p) >> 3);
  if (e.bias) {
#pragma unroll
    for (int h = 0; h < N / 8; ++h) {
      if (h < groups) {
        float b[8];
        load8(e.bias, e.bias_f32, p + 8 * h, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] += b[i];
      }
    }
  }
  uint32_t w[W];
  if (e.pre) {
    if constexpr (F32) {  // half a box of bf16: straight out
      if (q < e.Q) {
#pragma unroll
        for (int h = 0; h < N / 8; ++h)
          if (h < groups) store8_bf16(e.pre + q * e.P + p + 8 * h, reinterpret_cast<float(&)[8]>(v[8 * h]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = pack2_bf16(v[2 * i], v[2 * i + 1]);
      store_box(stage, lane, w, tpre, (int)p, (int)q0);
    }
  }
  act_all<N>(v, e.act);
  if (e.residual && q < e.Q) {
#pragma unroll
    for (int h = 0; h < N / 8; ++h) {
      if (h < groups) {
        float r[8];
        load8(e.residual, e.res_f32, q * e.P + p + 8 * h, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] += r[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = F32 ? __float_as_uint(v[i]) : pack2_bf16(v[2 * i], v[2 * i + 1]);
  store_box(stage, lane, w, tout, (int)p, (int)q0);
}

template <bool A_MN, bool B_MN, bool F32, bool KEEP>
__global__ void __launch_bounds__(kLinThreads, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                        const __grid_constant__ CUtensorMap tout, const __grid_constant__ CUtensorMap tpre,
                        const PairP p) {
  extern __shared__ unsigned char dyn[];
  __shared__ uint64_t full[kMaxRing], empty[kMaxRing], tfull[2], tempty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  unsigned char* ring = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int units = 2 * p.tq * p.tp - p.whole;
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    s_abort = 0;
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_mbar_init();
    prefetch_tmap(&ta);
    prefetch_tmap(&tb);
  } else if (warp == 1) {
    tmem_alloc_pair(&s_tmem, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    // -------------------------------------------------------------- producer --
    // Both CTAs' copies of a stage count on the first CTA's barrier.
    int s = 0;
    uint32_t ph = 0, armed = 0, armed_ph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += stride) {
      int a0, b0, half;
      pair_unit(p, u, a0, b0, half);
      if (half == 0) continue;
      a0 += (int)rank * 128;
      b0 += (int)rank * half;
      const uint32_t bytes = 2 * (kTileP * 128 + half * 128);
      for (int k = 0; k < p.steps; ++k) {
        if (!(ok = warp_wait(&empty[s], ph ^ 1, &s_abort))) break;
        if (elect_one()) {
          unsigned char* a = ring + (size_t)s * p.stage_bytes;
          unsigned char* b = a + kTileP * 128;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t bar = cluster_addr(smem_u32(&full[s]), 0);
          if (A_MN) {
            for (int i = 0; i < 2; ++i) tma_load_2d_pair(a + i * kBoxBytes, &ta, bar, a0 + 64 * i, k * kStepK);
          } else {
            tma_load_2d_pair(a, &ta, bar, k * kStepK, a0);
          }
          for (int i = 0; i < half; i += 64) {
            if (B_MN) tma_load_2d_pair(b + i * 128, &tb, bar, b0 + i, k * kStepK);
            else tma_load_2d_pair(b + i * 128, &tb, bar, k * kStepK, b0 + i);
          }
        }
        armed |= 1u << s;
        armed_ph = (armed_ph & ~(1u << s)) | (ph << s);
        if (++s == p.ring) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (ok) ok = __all_sync(0xffffffffu, producer_tail(empty, p.ring, s, ph, &s_abort));
    if (!ok) {
      if (lane == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
      if (rank == 0) drain_armed(full, p.ring, armed, armed_ph);
      // copies of the pair's other CTA that no barrier of this one was armed for
      const long long t0 = clock64();
      while (clock64() - t0 < (1 << 21)) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer --
    if (rank == 0) {
      int s = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      bool ok = true, issued = false;
      for (int u = first; ok && u < units; u += stride) {
        int q, c, half, n = 0;
        pair_unit(p, u, q, c, half);
        if (half == 0) continue;
        const uint32_t idesc = make_idesc_major(256, 2 * half, A_MN, B_MN);
        for (int k = 0; k < p.steps; ++k) {
          if (n == 0) {
            if (!(ok = warp_wait(&tempty[buf], bph ^ 1, &s_abort))) break;
            tc_fence_after();
          }
          if (!(ok = warp_wait(&full[s], ph, &s_abort))) break;
          tc_fence_after();
          const uint32_t a = smem_u32(ring + (size_t)s * p.stage_bytes), b = a + kTileP * 128;
          const bool last = k + 1 == p.steps || (KEEP && n + 1 == p.seg);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = A_MN ? sw128_mn_desc(a + kk * 2048, 64) : sw128_desc(a + kk * 32);
              const uint64_t bd = B_MN ? sw128_mn_desc(b + kk * 2048, 64) : sw128_desc(b + kk * 32);
              mma_bf16_pair(tmem + buf * 256, ad, bd, idesc, (n | kk) ? 1u : 0u);
            }
            mma_commit_pair(&empty[s], 3);
            if (last) mma_commit_pair(&tfull[buf], 3);
          }
          issued = true;
          if (++s == p.ring) {
            s = 0;
            ph ^= 1;
          }
          ++n;
          if (last) {
            n = 0;
            if (++buf == 2) {
              buf = 0;
              bph ^= 1;
            }
          }
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, accumulator_tail(tempty, buf, bph, &s_abort));
      if (!ok) {
        if (lane == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
        if (issued) {
          if (elect_one()) mma_commit_pair(&drain, 3);
          __syncwarp();
          const long long t0 = clock64();
          while (!mbar_try_wait(&drain, 0) && clock64() - t0 < kSpinLimitCycles) {
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue --
    constexpr int N = pair_box(F32, KEEP);
    const int quarter = warp & 3, side = (warp - 2) >> 2;
    unsigned char* stage = ring + (size_t)p.ring * p.stage_bytes + (warp - 2) * kStoreBytes;
    const uint32_t lead0 = cluster_addr(smem_u32(&tempty[0]), 0), lead1 = cluster_addr(smem_u32(&tempty[1]), 0);
    int buf = 0;
    uint32_t bph = 0;
    bool ok = true;
    for (int u = first; ok && u < units; u += stride) {
      int q, c, half;
      pair_unit(p, u, q, c, half);
      if (half == 0) continue;
      const int64_t q0 = (int64_t)q + rank * 128 + quarter * 32;
      const int64_t c0 = (int64_t)c + side * half;
      const uint32_t col = side * half + ((uint32_t)(quarter * 32) << 16);
      const bool rows = q0 < p.e.Q;
      if constexpr (KEEP) {
        float acc[128];
        for (int k = 0; k < p.steps; k += p.seg) {
          if (!(ok = warp_wait(&tfull[buf], bph, &s_abort))) break;
          tc_fence_after();
          const uint32_t at = tmem + buf * 256 + col;
#pragma unroll
          for (int i = 0; i < 128; i += 16) {
            if (i < half) {
              float v[16];
              tmem_ld16(at + i, v);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[i + j] = k == 0 ? v[j] : acc[i + j] + v[j];
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) cluster_mbar_arrive(buf ? lead1 : lead0);
          if (++buf == 2) {
            buf = 0;
            bph ^= 1;
          }
        }
        if (ok && rows) {
#pragma unroll
          for (int i = 0; i < 128; i += N)
            if (i < half && c0 + i < p.e.P)
              epilogue_box<F32, N>(p.e, q0 + lane, q0, c0 + i, acc + i, stage, lane, &tout, &tpre);
        }
      } else {
        if (!(ok = warp_wait(&tfull[buf], bph, &s_abort))) break;
        tc_fence_after();
        const uint32_t at = tmem + buf * 256 + col;
#pragma unroll 1
        for (int i = 0; i < half; i += N) {
          float v[N];
#pragma unroll
          for (int j = 0; j < N; j += 32) tmem_ld32(at + i + j, v + j);
          tmem_ld_wait();
          if (i + N >= half) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cluster_mbar_arrive(buf ? lead1 : lead0);
          }
          if (rows && c0 + i < p.e.P)
            epilogue_box<F32, N>(p.e, q0 + lane, q0, c0 + i, v, stage, lane, &tout, &tpre);
        }
        if (++buf == 2) {
          buf = 0;
          bph ^= 1;
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    if (!ok && lane == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no copy, product or arrival of the pair is left
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// --------------------------------------------------------- activation gradient --
// A CTA takes 64 x 8 columns and a share of the rows: thread (x, y) of 64 x 4 the
// columns 8 x .. 8 x + 7 of rows y, y + 4, ..., four of them (two of fp32) on their way at
// a time; the column sums of the CTA go to row blockIdx.y of the partial sums.
constexpr int kActCtas = 3;  // per SM

template <int ACT, bool DF32>
__global__ void __launch_bounds__(256, kActCtas) act_grad_kernel(const ActGradArgs a, int rows_per) {
  __shared__ float red[4][64][9];
  pdl_trigger();
  pdl_wait();
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int64_t c = ((int64_t)blockIdx.x * 64 + x) * 8;
  const int64_t m0 = (int64_t)blockIdx.y * rows_per;
  const int64_t m1 = m0 + rows_per < a.M ? m0 + rows_per : a.M;
  float s[8] = {};
  if (c < a.N) {
    constexpr int W = DF32 ? 2 : 1, kActRows = DF32 ? 2 : 4;
    for (int64_t m = m0 + y; m < m1; m += 4 * kActRows) {
      uint4 d[kActRows][W], z[kActRows];
#pragma unroll
      for (int r = 0; r < kActRows; ++r) {
        if (m + 4 * r < m1) {
          const int64_t at = (m + 4 * r) * a.N + c;
          const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(a.dout) + at * (DF32 ? 4 : 2));
#pragma unroll
          for (int i = 0; i < W; ++i) d[r][i] = from[i];
          if (ACT != kActNone) z[r] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.pre) + at);
        }
      }
#pragma unroll
      for (int r = 0; r < kActRows; ++r) {
        if (m + 4 * r >= m1) break;
        float f[8];
        if constexpr (DF32) {
          f[0] = __uint_as_float(d[r][0].x); f[1] = __uint_as_float(d[r][0].y);
          f[2] = __uint_as_float(d[r][0].z); f[3] = __uint_as_float(d[r][0].w);
          f[4] = __uint_as_float(d[r][1].x); f[5] = __uint_as_float(d[r][1].y);
          f[6] = __uint_as_float(d[r][1].z); f[7] = __uint_as_float(d[r][1].w);
        } else {
          unpack8_bf16(d[r][0], f);
        }
        if (ACT != kActNone) {
          float v[8];
          unpack8_bf16(z[r], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= act_slope(v[i], ACT);
        }
        if (a.dpre) store8_bf16(static_cast<bf16*>(a.dpre) + (m + 4 * r) * a.N + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += f[i];
      }
    }
  }
  if (!a.db) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[y][x][i] = s[i];
  __syncthreads();
  if (y != 0 || c >= a.N) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = ((red[0][x][i] + red[1][x][i]) + red[2][x][i]) + red[3][x][i];
  store8(a.part, true, (size_t)((int64_t)blockIdx.y * a.N + c), s);
}

// ------------------------------------------------------------------ host --
// Map of an operand: K-major [rows, K] in boxes of 64 K x box_rows, or MN-major
// [K, rows] in boxes of 64 rows x 64 K.
bool operand_map(CUtensorMap* m, const void* base, bool mn, int64_t rows, int64_t K, int box_rows) {
  return mn ? encode_map(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, K, rows, 64, kStepK,
                         CU_TENSOR_MAP_SWIZZLE_128B)
            : encode_map(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, K, kStepK, box_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int cluster, size_t smem, cudaStream_t st,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

constexpr int kSmemMax = 226 * 1024 - 1024;  // dynamic; the static part and the reserve beside it

// One instance of the split kernel: how many of its clusters of S CTAs run at once on a device (the
// current one), and its launch.
struct SplitForm {
  int (*clusters)(int device, int S);
  cudaError_t (*launch)(const ProductArgs& a, const Epi& e, int S, int steps, int seg, int* status, cudaStream_t st);
};

template <bool A_MN, bool B_MN, int BN>
struct Split {
  static constexpr int kPerSm = BN <= 64 ? 2 : 1;  // CTAs
  static constexpr int kStage = kTileP * 128 + (B_MN ? (BN + 63) / 64 * kBoxBytes : BN * 128);
  static constexpr int kRoom = (kPerSm == 2 ? kSmemMax / 2 - 2048 : kSmemMax) - 1024;
  static constexpr int kRing = kRoom / kStage < kMaxRing ? kRoom / kStage : kMaxRing;
  static constexpr size_t kSmem = (size_t)kRing * kStage + 1024;
  static_assert((size_t)kRing * kStage >= (size_t)BN * kTileP * 4, "the fp32 tile lies over the ring");
  // No allocation of TMEM waits for a CTA that waits for another: what fits on an SM together never wants
  // more than its 512 columns.  (The library's kernels that allocate all 512 have 145 KB of its 228.)
  static_assert(kPerSm * 2 * (BN < 32 ? 32 : BN) <= 512 && kSmem + (145 << 10) > (228 << 10) &&
                    (kPerSm + 1) * kSmem > (228 << 10),
                "tensor memory of the CTAs that share an SM");

  static auto kernel() { return product_split_kernel<A_MN, B_MN, BN>; }

  static int clusters(int device, int S) {
    static DeviceCounts<kMaxSplit + 1> known;
    return known.get(device, S, [S] {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = S;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(S);
      cfg.blockDim = dim3(kLinThreads);
      cfg.dynamicSmemBytes = kSmem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      cudaError_t e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel(), &cfg);
      if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return e == cudaErrorInvalidClusterSize ? 0 : -1;
      }
      // the query counts one CTA of a kernel with TMEM per SM; two run (at BN = 16, 256 CTAs take
      // the time of one round: 9.9 us)
      return n * kPerSm;
    });
  }

  static cudaError_t launch(const ProductArgs& a, const Epi& e, int S, int steps, int seg, int* status,
                            cudaStream_t st) {
    CUtensorMap ta, tb;
    if (!operand_map(&ta, a.a, A_MN, a.P, a.K, kTileP) || !operand_map(&tb, a.b, B_MN, a.Q, a.K, BN))
      return cudaErrorInvalidValue;
    SplitP p{};
    p.e = e;
    p.steps = steps;
    p.seg = seg;
    p.status = status;
    p.stage_bytes = kStage;
    p.ring = kRing;
    cudaError_t rc = cudaFuncSetAttribute(kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (rc == cudaSuccess && S > 8) rc = cudaFuncSetAttribute(kernel(), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (rc != cudaSuccess) return rc;
    const dim3 grid(S, (unsigned)((a.P + kTileP - 1) / kTileP), (unsigned)((a.Q + BN - 1) / BN));
    return launch_cluster(kernel(), grid, S, kSmem, st, ta, tb, p);
  }

  static SplitForm form() { return {&clusters, &launch}; }
};

template <bool A_MN, bool B_MN>
SplitForm split_form(int bn) {
  if constexpr (!B_MN) {
    if (bn == 16) return Split<A_MN, B_MN, 16>::form();
    if (bn == 32) return Split<A_MN, B_MN, 32>::form();
  }
  if (bn <= 64) return Split<A_MN, B_MN, 64>::form();
  if (bn == 128) return Split<A_MN, B_MN, 128>::form();
  return Split<A_MN, B_MN, 256>::form();
}

// Time of a split in us: rounds of clusters, each with a start and an end beside the stages of
// a part; a stage takes longer beside many other CTAs (they share L2), and where two are on
// an SM its loads bound it, 105 bytes a ns.  `least` is the time of the operands from memory.
// Against 5000 times of 270 products it picks one 1.5% above the best: us with the widest tile and clusters of up
// to eight, the best, and its BN and S: 512 x 1024 x 1024 9.3 7.4 64 4; 64 x 256 x 8192 9.6 7.4 32 16;
// 128 x 256 x 256 5.2 3.9 16 2; 256 x 4096 x 4096 15.6 15.6 256 4; dW 256 x 256 over 65536 rows 54 28 128 16.
double split_us(int bn, int64_t tiles, int at_once, int S, int steps, int sms, double least) {
  const double ends = (bn == 16 ? 3.45 : (bn == 32 ? 4.0 : (bn == 64 ? 4.9 : (bn == 128 ? 5.3 : 7.5)))) +
                      (S > 1 ? 0.05 : 0.0) + (S > 8 ? 0.3 : 0.0) + 0.01 * S;
  const int64_t rounds = (tiles + at_once - 1) / at_once;
  const double ctas = (double)(tiles < at_once ? tiles : at_once) * S;
  double stage = (bn == 256 ? 0.33 : 0.275) * (1 + 0.4 * (ctas < 32 ? 0.0 : (ctas > 96 ? 1.0 : (ctas - 32) / 64)));
  const double loads = 2 * (kTileP + bn) * kStepK * 2 / 105e3;
  if (ctas > sms && stage < loads) stage = loads;
  const double us = rounds * ((steps + S - 1) / S) * stage;
  return (us > least ? us : least) + rounds * ends;
}

// Tiles of 256 x 256 that the pairs take whole: where half of the pairs or more would idle
// in the last round, its tiles are split in two.
int pair_whole(int64_t tiles, int pairs) {
  const int64_t rest = tiles % pairs;
  return (int)(2 * rest <= pairs ? tiles - rest : tiles);
}

template <bool A_MN, bool B_MN, bool F32, bool KEEP>
cudaError_t launch_pair(const ProductArgs& a, const Epi& e, int steps, int sms, int* status, cudaStream_t st) {
  CUtensorMap ta, tb, to, tp;  // the pair's rows are q (b of the product), its columns p (a)
  constexpr int box = pair_box(F32, KEEP);
  constexpr auto swizzle = F32 || !KEEP ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_32B;
  const auto out_type = F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!operand_map(&ta, a.b, A_MN, a.Q, a.K, kTileP) || !operand_map(&tb, a.a, B_MN, a.P, a.K, 64) ||
      !encode_map(&to, a.out, out_type, F32 ? 4 : 2, a.Q, a.P, box, 32, swizzle) ||
      !encode_map(&tp, a.pre ? a.pre : a.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.Q, a.P, F32 ? 64 : box, 32,
                  F32 ? CU_TENSOR_MAP_SWIZZLE_128B : swizzle))
    return cudaErrorInvalidValue;
  const int64_t tiles = (a.Q + 255) / 256 * ((a.P + 255) / 256);
  PairP p{};
  p.e = e;
  p.steps = steps;
  p.tq = (int)((a.Q + 255) / 256);
  p.tp = (int)((a.P + 255) / 256);
  p.whole = pair_whole(tiles, sms / 2);
  p.group = 8;
  p.seg = F32 ? kSegSteps : kLongSeg;
  p.status = status;
  p.stage_bytes = 2 * kTileP * 128;
  p.ring = (kSmemMax - 1024 - kEpiWarps * kStoreBytes) / p.stage_bytes;
  auto kern = product_pair_kernel<A_MN, B_MN, F32, KEEP>;
  cudaError_t rc = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (rc != cudaSuccess) return rc;
  const int64_t units = 2 * tiles - p.whole;
  const int pairs = units < sms / 2 ? (int)units : sms / 2;
  return launch_cluster(kern, dim3(2 * pairs), 2,
                        (size_t)p.ring * p.stage_bytes + kEpiWarps * kStoreBytes + 1024, st, ta, tb, to, tp, p);
}

}  // namespace

bool linear_form(const char* name, LinearForm* form) {
  static const struct {
    const char* name;
    LinearForm form;
  } forms[] = {{"", kFormAuto}, {"token", kFormToken}, {"split", kFormSplit}, {"pair", kFormPair}};
  for (const auto& f : forms)
    if (strcmp(name ? name : "", f.name) == 0) {
      *form = f.form;
      return true;
    }
  return false;
}

cudaError_t launch_product(const ProductArgs& a, int sms, int* status, cudaStream_t st) {
  Epi e{};
  e.bias = a.bias;
  e.residual = a.residual;
  e.pre = static_cast<bf16*>(a.pre);
  e.out = a.out;
  e.act = a.act;
  e.bias_f32 = a.bias_f32;
  e.res_f32 = a.res_f32;
  e.out_f32 = a.out_f32;
  e.P = a.P;
  e.Q = a.Q;
  if (!a.a_mn && !a.b_mn && a.Q == 1 && (a.form == kFormAuto || a.form == kFormToken)) {
    int W = 1;  // warps per row: enough of them to fill the SMs, two loads for each at least
    while (W < kRowsWarps && a.P / kRowsR * W < (int64_t)sms * 48 && a.K / 8 > 64 * W) W *= 2;
    const int64_t per = kRowsWarps / W * kRowsR;
    return launch_kernel(product_token_kernel, dim3((unsigned)((a.P + per - 1) / per)), dim3(kRowsWarps * 32), 0, st,
                         static_cast<const bf16*>(a.a), static_cast<const bf16*>(a.b), a.K, W, e);
  }
  const int steps = (int)((a.K + kStepK - 1) / kStepK);
  int device = 0;
  const cudaError_t rc = cudaGetDevice(&device);
  if (rc != cudaSuccess) return rc;
  int S = 0;
  double best = 0;
  SplitForm split{};
  const double least = (double)(a.P + a.Q) * a.K * 2 / 6.8e6;
  int widest = 16;
  while (widest < a.Q && widest < 256) widest *= 2;
  for (int bn = a.b_mn && widest < 64 ? 64 : widest; bn >= (a.b_mn ? 64 : 16); bn /= 2) {
    const SplitForm f = a.a_mn ? (a.b_mn ? split_form<true, true>(bn) : split_form<true, false>(bn))
                               : split_form<false, false>(bn);
    const int64_t tiles = (a.P + kTileP - 1) / kTileP * ((a.Q + bn - 1) / bn);
    if ((a.Q + bn - 1) / bn > 65535) break;
    for (int s = 1; s <= kMaxSplit && s <= steps; s += s < 8 ? 1 : 8) {
      const int at_once = f.clusters(device, s);
      if (at_once < 1) continue;
      const double us = split_us(bn, tiles, at_once, s, steps, sms, least);
      if (S == 0 || us < best) {
        best = us;
        S = s;
        split = f;
      }
    }
  }
  // The pairs' time, likewise: rounds of whole and of half tiles, none shorter than its
  // epilogue.  256 x 4096 x 64 4.9 us, 512 x 4096 x 4096 22.6 (halves), 700 x 4096 x 2048 15.9,
  // 1024 x 4096 x 4096 25.4, 4096 x 12288 x 64 29.8; split 4.8, 21.3, 19.8, 32.4, 87.
  const int64_t pt = (a.Q + 255) / 256 * ((a.P + 255) / 256);
  const int pairs = sms / 2;
  const int64_t whole = pair_whole(pt, pairs), halves = 2 * (pt - whole);
  auto round = [&](double stage) { return steps * stage > 2.3 ? steps * stage : 2.3; };
  const double pair_us = 2.4 + (steps < 7 ? 0.3 * steps : 2.0) + round(0.31) * ((whole + pairs - 1) / pairs) +
                         round(0.255) * ((halves + pairs - 1) / pairs);
  const bool pair = S == 0 || (a.form == kFormAuto ? pair_us < best : a.form == kFormPair);
  if (pair) {
    const bool keep = steps > (a.out_f32 ? kSegSteps : kLongSteps);
#define MOE_PAIR(A, B, F32)                                                    \
  return keep ? launch_pair<A, B, F32, true>(a, e, steps, sms, status, st)     \
              : launch_pair<A, B, F32, false>(a, e, steps, sms, status, st)
    if (a.a_mn && a.b_mn) {
      if (a.out_f32) MOE_PAIR(true, true, true);
      MOE_PAIR(true, true, false);
    }
    if (a.a_mn) MOE_PAIR(false, true, false);  // (dx is bf16)
    if (a.out_f32) MOE_PAIR(false, false, true);
    MOE_PAIR(false, false, false);
#undef MOE_PAIR
  }
  const int seg = a.out_f32 ? kSegSteps : ((steps + S - 1) / S > kLongSteps ? kLongSeg : 1 << 30);
  return split.launch(a, e, S, steps, seg, status, st);
}

cudaError_t launch_act_grad(const ActGradArgs& a, int sms, cudaStream_t st) {
  // row shares: one round of CTAs
  const int64_t strips = (a.N + 511) / 512;
  int64_t shares = kActCtas * sms / strips;
  if (shares > (a.M + 15) / 16) shares = (a.M + 15) / 16;
  if (shares > kActGradRows) shares = kActGradRows;
  if (shares < 1) shares = 1;
  const int rows_per = (int)((a.M + shares - 1) / shares);
  if (a.M > 0) shares = (a.M + rows_per - 1) / rows_per;
  else shares = 0;
  if (shares > 0) {
    auto kern = act_grad_kernel<kActNone, false>;
#define MOE_ACT(A) \
  if (a.act == A) kern = a.dout_f32 ? act_grad_kernel<A, true> : act_grad_kernel<A, false>
    MOE_ACT(kActNone);
    MOE_ACT(kActRelu);
    MOE_ACT(kActSilu);
    MOE_ACT(kActGelu);
    MOE_ACT(kActGeluTanh);
#undef MOE_ACT
    cudaError_t e = launch_kernel(kern, dim3((unsigned)strips, (unsigned)shares), dim3(256), 0, st, a,
                                  rows_per);
    if (e != cudaSuccess) return e;
  }
  if (!a.db) return cudaSuccess;
  return launch_column_sum(a.part, (int)shares, a.N, a.N, a.N, a.db, nullptr, sms, st);
}

}  // namespace moe
