// moe_layer_forward: the whole MoE block for a few tokens (T <= 8) in two
// launches.
//
//   x_hat = x r (.) w,  r = 1 / sqrt(mean(x^2) + eps)
//   logits = x_hat W_r + b; top-k; softmax over the k
//   a = silu(x_hat Wg^T) (.) (x_hat Wu^T);  f = sum_j w_j (a W2^T);  tail(f)
//
// With T <= 8 tokens the time is the expert weights' way through HBM once
// (8 experts of 38 MB at T = 1, H = 4096, I = 1536, top_k = 8: 45 us); all else
// has to hide behind it.
//
// Launch 1 (layer_route_kernel) multiplies x by the norm weight, writes it in the
// form the products take, and takes the router's partial dot products and the
// partial sums of squares per K chunk.  r is a factor of the row, so it is
// applied afterwards, to the logits and to the FC1 results, and nothing in this
// launch waits for a whole row.
//
// Launch 2 (layer_experts_kernel), one persistent CTA per SM: every CTA adds the
// partial logits and picks the experts by itself, takes FC1 row tiles of the
// active experts from a counter, waits until all tiles are done, and computes
// its own slice of H output rows over all experts -- the sum over a token's
// experts stays in its accumulators.  The CTAs that finish last do the tail.
// Claiming the FC1 tiles from a counter means the wait needs no co-residency:
// a CTA that has not started holds no tile.
//
// Products: the weights are the 16 x 16 operand of m16n8k16 MMAs with fp32
// accumulation; the 8 columns are the tokens' activations in two 16-bit terms
// hi + lo, so that neither x_hat nor the intermediate is rounded to 16 bits.  With
// T <= 4 both terms of a token fit one MMA's columns.
//   bf16 weights  bf16 terms (16 bits of mantissa)
//   E4M3 weights  fp16 terms (22 bits): E4M3 -> fp16 is exact and one instruction
//                 for two weights, E4M3 -> bf16 four.  fp16 has little range, so
//                 the terms carry powers of two: a token's 128 columns of x share
//                 one, applied with the weight scale after a step; eight columns
//                 of the intermediate do (a row tile, all that a claim is sure to
//                 hold of them), brought by an fp16 product to the largest among the
//                 step's 128 columns when they are used.  So a value is held to
//                 2^-22 of itself or 2^-38 of the largest of its 128 columns,
//                 whichever is more (fp16 steps end at 2^-24, the largest is
//                 above 2^14), and a large column takes nothing from those of other
//                 steps.  (mma.sync on E4M3 itself is no way
//                 around the conversion: it runs as one, 51 cycles per m16n8k32
//                 against 22 per m16n8k16 with operands from shared memory.)
//
// Sixteen warps: eight consumers, each with a producer warp of its own that fills
// the consumer's part of shared memory a few steps ahead (cp.async; a pair of
// mbarriers per step).  The pieces lie as the consumer's lanes feed them to the
// MMAs, so a step is 16-byte shared loads, conversions and MMAs and nothing else
// (with the copies issued by the same warps: 119 us against 113 for four tokens
// with block-wise FP8).  The order of the K elements inside a piece is the same for
// both operands and therefore free.  The activations go the same way as the
// weights: a plain load of them would wait behind the copies in flight (8 tokens
// 375 us against 256).  The first W2 pieces are on their way while the CTA waits
// for the other CTAs' FC1 tiles.
//
// mma.sync and not tcgen05: with 8 columns the tensor pipe is 8 to 20% busy and
// HBM is what binds; a fragment read straight from the copied bytes needs no
// descriptor layout, row tiles of 16 let every CTA have an equal share of the
// output rows (27 of 4096), and accumulators in registers spare the TMEM round
// trip between tiles that short.
//
// Measured (H = 4096, I = 1536, E = 64, top_k = 8, cold weights): one token 61.7 us
// (302 MB), eight tokens 250 us (1.775 GB read, 7.1 TB/s), E4M3 one token 33.5 us,
// block-wise FP8 four tokens 94 us (5.0 TB/s).  The separate launches of
// moe_ffn_forward, without a tail: 96, 251, 54 and 122 us.  What is left at one token
// is latency around the stream: the routing launch 3 to 4 us, the hand-over 1, the
// routing in each CTA 3, the wait between FC1 and FC2 2 to 3, the tail 3 to 4.
#include "block_tail.cuh"
#include "kernels.h"
#include "tail.h"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

#include <stddef.h>

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsL = 32 * kWarps;  // consumers; as many producers follow them

// TOK: tokens that the columns have room for (T <= TOK).  Column c of MMA j holds
// term j * kTpg + c % kTpg of token c / kTpg.
template <int TOK>
struct Cols {
  static constexpr int kTpg = 8 / TOK;     // terms of a token per MMA
  static constexpr int kMmas = 2 / kTpg;   // MMAs per weight tile and K
};

// Per-warp stage of the copy ring: weights [2 tiles][2 row halves][2 K blocks]
// [32 lanes] of 16 bytes; activations [2 K blocks][MMAs][pieces][32 lanes] of 16
// bytes; FP8: the scales of the 32 rows and the powers of two of the tokens.
constexpr int kStepA = 4096;
template <bool FP8, int TOK>
struct Ring {
  static constexpr int kPieces = FP8 ? 2 : 1;  // of one term for 16 bytes of weights
  static constexpr int kScaleAt = kStepA + 2 * Cols<TOK>::kMmas * kPieces * 512;
  static constexpr int kPowAt = kScaleAt + 128;
  static constexpr int kStage = kScaleAt + (FP8 ? 128 + 2 * TOK * 8 : 0);
  static constexpr int kDepth = (200 << 10) / (kWarps * kStage);  // 3 .. 5 steps
  static constexpr int kWarp = kDepth * kStage;
  static constexpr int kBytes = kWarps * kWarp;
};
constexpr int kRed = kWarps * 2 * 16 * 8;  // floats: partial sums of all warps, two row tiles
constexpr int kMaxPairs = kLayerMaxT * kMaxTopK;
constexpr int kCtrInts = 3;

struct LayerP {
  const bf16* x;
  const bf16* norm_w;
  const float* router_w;
  const float* logits;
  const float* bias;
  const int32_t* ids_in;
  const float* tw_in;
  const void* w13;
  const void* w2;
  const float* s13;
  const float* s2;
  int32_t* ids_out;
  float* tw_out;
  void* out;  // bf16 [T, H] without a tail
  int T, H, E, I, k, block_scales;
  float eps;
  // workspace
  uint16_t* xt;        // terms of x w [2][T, H], bf16 or (FP8) fp16
  uint16_t* at;        // terms of the intermediate [2][T k, I], times the routing weight
  float* xpow;         // FP8: powers of two of x w [T, H / 128]
  uint8_t* apow;       // FP8: exponents (pow_exponent) of the intermediate's 8-column groups [T k, I / 8]
  float *ssq, *part;   // sums of squares [chunks, 8], partial logits [chunks, T, E]
  float* f;            // [T, H]
  int* ctr;            // [0] FC1 claims, [1] FC1 tiles done, [2] CTAs finished
  int* status;
};

// K chunk c covers the units [c n / 16, (c + 1) n / 16) of 128 columns (the last
// unit may be 64 wide).
struct Chunk {
  int k0, k1;
};
__host__ __device__ inline Chunk layer_chunk(int H, int c) {
  const int n = (H + 127) >> 7;
  Chunk ch;
  ch.k0 = c * n / kLayerChunks * 128;
  ch.k1 = (c + 1) * n / kLayerChunks * 128;
  if (ch.k1 > H) ch.k1 = H;
  return ch;
}

// v in two 16-bit terms.
template <bool F16>
MOE_DEV void split16(float v, uint16_t& hi, uint16_t& lo) {
  if (F16) {
    const __half h = __float2half_rn(v);
    hi = __half_as_ushort(h);
    lo = __half_as_ushort(__float2half_rn(v - __half2float(h)));
  } else {
    const bf16 h = __float2bfloat16_rn(v);
    hi = __bfloat16_as_ushort(h);
    lo = __bfloat16_as_ushort(__float2bfloat16_rn(v - __bfloat162float(h)));
  }
}

// fp16 terms: values of which the largest magnitude m has the biased exponent e
// are scaled by 2^(141 - e), to below 2^15, and the products by 2^(e - 141).
// Magnitudes below 2^-112 count as that; infinities and NaN stay what they are.
MOE_DEV int pow_exponent(float m) {
  const int e = (int)((__float_as_uint(m) >> 23) & 255u);
  return e < 15 ? 15 : (e > 254 ? 254 : e);
}
MOE_DEV float pow_up(int e) { return __uint_as_float((uint32_t)(268 - e) << 23); }
MOE_DEV float pow_down(int e) { return __uint_as_float((uint32_t)(e - 14) << 23); }

// ------------------------------------------------------------------ launch 1 --
// Grid (kLayerChunks, groups of 32 experts): K chunk c, experts 32y .. 32y+31; TT:
// tokens that the dot products have room for (T <= TT).  Latency is all there is:
// the chunk of x and each warp's rows of W_r (16 at H = 4096) are on their way
// before anything is waited for.
constexpr int kRouteWarps = 16;

template <bool FP8, int TT>
__global__ void __launch_bounds__(32 * kRouteWarps) layer_route_kernel(const LayerP p) {
  extern __shared__ __align__(16) float xw[];  // [rows of the chunk][TT tokens]
  __shared__ float red[kRouteWarps][TT][32];
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x;
  const Chunk ch = layer_chunk(p.H, c);
  const int k0 = ch.k0, rows = ch.k1 - ch.k0;
  const int e = blockIdx.y * 32 + lane;
  const float* wr = p.router_w ? p.router_w + (size_t)k0 * p.E + e : nullptr;
  // One warp runs the code twice: first, while the others already wait for the work in
  // front of this launch, without touching what they share, for the instructions to be
  // at hand afterwards (on the SMs that get these CTAs they rarely are: one token 1 us
  // of 62, two tokens at H = 7168 1.5 of 201).  The first time it reads shared memory that
  // nobody has written yet or that the others, further ahead, are writing: that race is
  // there on purpose, what it reads and computes goes nowhere but into its own part of
  // `red`, which it writes again before anyone reads it.
  int live = warp != kRouteWarps - 1;
  asm volatile("" : "+r"(live));
#pragma unroll 1
  for (;; live = 1) {
    if (live) pdl_wait();
    const int t0 = live ? warp : 0;
    const bool on = t0 < p.T;  // warp t: token t (zeros beyond the last)
    const int nv = (live ? rows : min(rows, 256)) >> 3;
    const size_t row = (size_t)(on ? t0 : 0) * p.H + k0;
    if (live && c == 0 && blockIdx.y == 0 && tid < kCtrInts) p.ctr[tid] = 0;
    // the first 256 columns of x and the norm's weights
    uint4 x0 = make_uint4(0u, 0u, 0u, 0u), w0 = x0;
    if (live && on && lane < nv) {
      x0 = *reinterpret_cast<const uint4*>(p.x + row + lane * 8);
      w0 = *reinterpret_cast<const uint4*>(p.norm_w + k0 + lane * 8);
    }
    constexpr int U = 16;
    float wv[U];
    if (wr) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = warp + kRouteWarps * u;
        wv[u] = (live && r < rows && e < p.E) ? wr[(size_t)r * p.E] : 0.f;
      }
    }
    if (t0 < TT) {
      float ss = 0.f;
#pragma unroll 1
      for (int v0 = 0; v0 < nv; v0 += 32) {
        const int v = v0 + lane;
        if (v0 && on && v < nv) {  // (live)
          x0 = *reinterpret_cast<const uint4*>(p.x + row + v * 8);
          w0 = *reinterpret_cast<const uint4*>(p.norm_w + k0 + v * 8);
        }
        float a[8] = {};
        if (on && v < nv) {
          float w[8];
          unpack8_bf16(x0, a);
          unpack8_bf16(w0, w);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            ss = fmaf(a[q], a[q], ss);
            a[q] *= w[q];
          }
        }
        if (live && wr && v < nv) {
#pragma unroll
          for (int q = 0; q < 8; ++q) xw[(v * 8 + q) * TT + warp] = a[q];
        }
        if (blockIdx.y == 0) {
          const size_t at = row + v * 8, term = (size_t)p.T * p.H;
          float up = 1.f;
          if (FP8) {  // 16 lanes share a power of two
            float m = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(a[q]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int ex = pow_exponent(m);
            up = pow_up(ex);
            if (live && on && v < nv && (lane & 15) == 0)
              p.xpow[warp * ((p.H + 127) >> 7) + ((k0 + v * 8) >> 7)] = pow_down(ex);
          }
          if (on && v < nv) {
            __align__(16) uint16_t hi[8], lo[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) split16<FP8>(a[q] * up, hi[q], lo[q]);
            if (live) {
              *reinterpret_cast<uint4*>(p.xt + at) = *reinterpret_cast<uint4*>(hi);
              *reinterpret_cast<uint4*>(p.xt + term + at) = *reinterpret_cast<uint4*>(lo);
            }
          }
        }
      }
      if (blockIdx.y == 0) {
        ss = warp_sum(ss);
        if (live && on && lane == 0) p.ssq[c * kLayerMaxT + warp] = ss;
      }
    }
    if (!wr) {
      if (live) return;
      continue;
    }
    if (live) __syncthreads();
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    for (int r0 = warp; r0 < nv * 8; r0 += kRouteWarps * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + kRouteWarps * u;
        if (r < rows) {
          float a[TT];
          if constexpr (TT % 4 == 0) {
#pragma unroll
            for (int t = 0; t < TT; t += 4) {
              const float4 q = *reinterpret_cast<const float4*>(&xw[r * TT + t]);
              a[t] = q.x; a[t + 1] = q.y; a[t + 2] = q.z; a[t + 3] = q.w;
            }
          } else {
            const float2 q = *reinterpret_cast<const float2*>(&xw[r * TT]);
            a[0] = q.x; a[1] = q.y;
          }
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[t] = fmaf(a[t], wv[u], acc[t]);
        }
        const int rn = r + kRouteWarps * U;
        wv[u] = (live && rn < rows && e < p.E) ? wr[(size_t)rn * p.E] : 0.f;
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) red[warp][t][lane] = acc[t];
    if (live) __syncthreads();
    if (on && e < p.E) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) s += red[w][t0][lane];
      if (live) p.part[((size_t)c * p.T + warp) * p.E + e] = s;
    }
    if (live) return;
  }
}

// ------------------------------------------------------------------ launch 2 --
MOE_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Through L1: activations.  Their pieces are parts of sectors that several copies
// and all steps of a claim share; past L1 each would be an L2 request of its own
// (FP8 one token 45.9 us against 35.5, four tokens 111 against 99).
MOE_DEV void cp_async16_l1(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Past L1, with `bytes` of 16 from src and the rest zeros.
MOE_DEV void cp_async16z(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrives on the barrier once this thread's copies so far have landed.
MOE_DEV void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}
MOE_DEV void cp_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MOE_DEV uint4 hmul2x4(const uint4& a, uint32_t b) {
  uint4 d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d.x) : "r"(a.x), "r"(b));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d.y) : "r"(a.y), "r"(b));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d.z) : "r"(a.z), "r"(b));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d.w) : "r"(a.w), "r"(b));
  return d;
}
MOE_DEV void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreadsL) : "memory"); }
MOE_DEV void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <bool F16>
MOE_DEV void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes as two fp16 pairs (exact).
MOE_DEV void e4m3x4_f16(uint32_t q, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(q));
}

constexpr int kMaxDepth = 5;

struct __align__(16) LayerSmem {
  int32_t ids[kLayerMaxT][kMaxTopK];
  float w[kLayerMaxT][kMaxTopK];
  float r[kLayerMaxT];
  unsigned used[kMaxExperts];  // tokens of each expert, as a bit mask
  int slot[kMaxExperts];       // its place among the active experts
  int expert[kMaxPairs];
  unsigned mask[kMaxPairs];
  __align__(16) int pair[kMaxPairs][kLayerMaxT];  // (written in 16-byte stores)
  float wt[kMaxPairs][kLayerMaxT];
  int warp_cnt[kWarps];
  int claim[4];
  int published;  // newest claim index in claim[]
  int fc1_done;
  int flag;
  int abort;
  int in_time;  // result of a wait, for all consumers
  float sum[kWarps];
  uint64_t full[kWarps][kMaxDepth], empty[kWarps][kMaxDepth];
};
static_assert(alignof(LayerSmem) == 16 && offsetof(LayerSmem, pair) % 16 == 0 &&
                  sizeof(LayerSmem::pair[0]) % 16 == 0,
              "16-byte stores to pair");

// A logit as a key of the top-k: its bits in an order-preserving form, NaN as -inf
// (0x007fffff), -0 as 0.  Keys of logits are above 0.
MOE_DEV unsigned order_key(float z) {
  z = (z != z) ? -INFINITY : z + 0.0f;
  const unsigned u = __float_as_uint(z);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The keys of the experts lane + 32 i of token t, 0 beyond E.  ss: this lane's part of
// the token's sum of squares.
template <int PER>
MOE_DEV void layer_keys(const LayerP& p, int t, int lane, float ss, unsigned (&key)[PER], float& r) {
  float zs[PER], bias[PER];  // every load is issued before the first use
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    zs[i] = bias[i] = 0.f;
    if (e < p.E) {
      if (p.bias) bias[i] = p.bias[e];
      if (p.logits) {
        zs[i] = p.logits[(size_t)t * p.E + e];
      } else {
        float part[kLayerChunks];
#pragma unroll
        for (int c = 0; c < kLayerChunks; ++c) part[c] = __ldcg(&p.part[((size_t)c * p.T + t) * p.E + e]);
#pragma unroll
        for (int c = 0; c < kLayerChunks; ++c) zs[i] += part[c];
      }
    }
  }
  r = 1.0f / sqrtf(warp_sum(ss) / (float)p.H + p.eps);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = 0;
    if (lane + 32 * i < p.E) {
      float z = p.logits ? zs[i] : zs[i] * r;
      if (p.bias) z += bias[i];
      key[i] = order_key(z);
    }
  }
}

// layer_keys of 32 experts (part `at`) for all warps; part: of chunk 0, `step` apart.
// (Not inlined: the steps' registers are all taken, and code beside them moves them.)
__device__ __noinline__ void layer_part(const float* logits, const float* part, const float* bias,
                                        const float* ssq, int step, int E, int H, float eps, int at,
                                        unsigned* keys, float* r_out) {
  const int lane = threadIdx.x & 31, e = at * 32 + lane;
  const float ss = lane < kLayerChunks ? __ldcg(&ssq[lane * kLayerMaxT]) : 0.f;
  float z = 0.f, b = 0.f;
  if (e < E) {
    if (bias) b = bias[e];
    if (logits) {
      z = logits[e];
    } else {
      float v[kLayerChunks];
#pragma unroll
      for (int c = 0; c < kLayerChunks; ++c) v[c] = __ldcg(&part[(size_t)c * step + e]);
#pragma unroll
      for (int c = 0; c < kLayerChunks; ++c) z += v[c];
    }
  }
  const float r = 1.0f / sqrtf(warp_sum(ss) / (float)H + eps);
  if (e < E) keys[e] = order_key((logits ? z : z * r) + b);
  if (e == 0) *r_out = r;
}

// Top-k of one token by one warp with the results of warp_topk (common.cuh):
// larger logit first, ties to the lower expert, NaN as -inf, softmax over the
// selected (summed in slot order), weights 0 when all of them are -inf.  Here
// the arg-max is two warp reductions of integers: the keys, then the lowest expert
// that has the maximum.  keys: where other warps have left them (and r), or NULL.
template <int PER>
MOE_DEV void layer_topk(const LayerP& p, int t, int lane, float ss, const unsigned* keys, LayerSmem* sm) {
  unsigned key[PER];  // 0: taken or beyond E
  if (PER > 2 && keys) {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = lane + 32 * i < p.E ? keys[lane + 32 * i] : 0u;
  } else {
    float r;
    layer_keys<PER>(p, t, lane, ss, key, r);
    if (lane == 0) sm->r[t] = r;
  }
  float mine = 0.f, top = 0.f, s = 0.f;
  int sel_e = 0;
  bool some = false;
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    unsigned m = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = max(m, key[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == m) at = lane + 32 * i;
    at = __reduce_min_sync(0xffffffffu, at);
    if ((at & 31u) == (unsigned)lane) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if ((int)(at >> 5) == i) key[i] = 0;
    }
    const float z = __uint_as_float((m & 0x80000000u) ? m & 0x7fffffffu : ~m);  // (every lane)
    if (j == 0) {
      top = z;
      some = z > -INFINITY;
    }
    const float e = some ? expf(z - top) : 0.f;
    s += e;
    if (lane == j) {
      mine = e;
      sel_e = (int)at;
    }
  }
  if (lane < p.k) {
    sm->ids[t][lane] = sel_e;
    sm->w[t][lane] = some ? mine / s : 0.f;
  }
}

// The tail (block_tail.cuh) of row t by the whole CTA.  `buf`: shared memory for
// the row's inputs, brought there by asynchronous copies that all run at once
// (what the tail reads was last touched before the weights went through L2), or
// nothing, when they do not fit.  The loops are kept short on purpose: this code
// runs once per launch, on T of the SMs, and its instructions come from wherever
// the weights' way through L2 has left them.  dry: one round of the loops on
// whatever `buf` holds, without a store to global memory (see the kernel).
MOE_DEV void layer_tail_row(const LayerP& p, const TailP& tail, int t, int grow, float factor,
                            unsigned char* buf, bool staged, float* red, bool dry) {
  const int tid = threadIdx.x, lane = tid & 31, H = p.H;
  const int nv = dry ? min(H >> 3, kThreadsL) : H >> 3;
  const size_t row = (size_t)t * H;
  const bool gate_row = tail.gate && tail.gate_cols != 1 && grow >= 0;
  float* f = reinterpret_cast<float*>(buf);  // [H], then h
  const unsigned char* s_res = buf + (size_t)H * 4;
  const unsigned char* s_gate = s_res + (size_t)H * 4;
  const unsigned char* s_pw = s_gate + (size_t)H * 4;
  const unsigned char* s_nw = s_pw + (size_t)H * 2;
  if (staged) cp_wait_all();
  if (!dry) consumer_sync();
  auto reduce = [&](float v, bool mx) {
    v = mx ? warp_max(v) : warp_sum(v);
    if (lane == 0) red[tid >> 5] = v;
    if (!dry) consumer_sync();
    v = red[0];
    for (int w = 1; w < kWarps; ++w) v = mx ? fmaxf(v, red[w]) : v + red[w];
    if (!dry) consumer_sync();
    return v;
  };
  float r = 1.f;
  if (tail.post_w) {
    float ss = 0.f;
#pragma unroll 1
    for (int v = tid; v < nv; v += kThreadsL) {
      float a[8];
      load8(f, true, v * 8, a);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(a[q], a[q], ss);
    }
    r = 1.0f / sqrtf(reduce(ss, false) / (float)H + tail.post_eps);
  }
  float ss = 0.f;
#pragma unroll 1
  for (int v = tid; v < nv; v += kThreadsL) {
    float a[8], w[8], res[8], h[8];
    load8(f, true, v * 8, a);
    if (tail.post_w) load8(staged ? (const void*)s_pw : tail.post_w, false, v * 8, w);
    if (tail.residual) {
      load8(staged ? s_res : tail.residual, tail.res_f32 != 0, staged ? (size_t)v * 8 : row + v * 8, res);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) res[q] = 0.f;
    }
    if (tail.post_w) {
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] = (a[q] * r) * w[q];
    }
    if (gate_row) {
      load8(staged ? s_gate : tail.gate, tail.gate_f32 != 0, staged ? (size_t)v * 8 : (size_t)grow * H + v * 8,
            w);
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] *= w[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      h[q] = grow >= 0 ? fmaf(factor, a[q], res[q]) : res[q];
      ss = fmaf(h[q], h[q], ss);
    }
    if (!dry) store8(tail.out, tail.out_f32 != 0, row + v * 8, h);
    float4* keep = reinterpret_cast<float4*>(f + v * 8);  // read back by this thread
    keep[0] = make_float4(h[0], h[1], h[2], h[3]);
    keep[1] = make_float4(h[4], h[5], h[6], h[7]);
  }
  if (!tail.next_w) return;
  const float rn = 1.0f / sqrtf(reduce(ss, false) / (float)H + tail.next_eps);
  float amax = 0.f, s = 1.f;
  // pass 0: x_hat, its maxima, codes per group; pass 1: codes per token
#pragma unroll 1
  for (int pass = 0; pass < (tail.xq && !tail.q_group ? 2 : 1); ++pass) {
    if (pass) {
      amax = reduce(amax, true);
      s = tail_scale(amax);
      if (tid == 0 && !dry) tail.xscale[t] = s;
    }
#pragma unroll 1
    for (int v0 = 0; v0 < nv; v0 += kThreadsL) {  // (whole warps: a group's maximum is a shuffle)
      const int v = v0 + tid;
      float a[8], w[8], m = 0.f;
      if (v < nv) {
        load8(f, true, v * 8, a);
        load8(staged ? (const void*)s_nw : tail.next_w, false, v * 8, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          a[q] = (a[q] * rn) * w[q];
          m = fmaxf(m, fabsf(a[q]));
        }
        if (!pass && tail.xhat && !dry) store8_bf16(tail.xhat + row + v * 8, a);
      }
      if (tail.q_group) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = tail_scale(m);
        if (tail.xq && v < nv && (v & 15) == 0 && !dry) tail.xscale[(size_t)t * (H >> 7) + (v >> 4)] = s;
      }
      amax = fmaxf(amax, m);
      if (tail.xq && v < nv && (pass || tail.q_group) && !dry)
        *reinterpret_cast<uint2*>(tail.xq + row + v * 8) = tail_e4m3x8(a, s);
    }
  }
}

// FP8: E4M3 weights, one scale per (row >> rs) and K step * ks.
// Returns the row of the tail that the CTA's consumers are to do, or -1.
template <bool FP8, int TOK>
MOE_DEV int layer_experts(const LayerP& p, int has_tail, unsigned char* ring_all, LayerSmem& sm,
                          float (&red)[2][kRed]) {
  constexpr int EB = FP8 ? 1 : 2;  // bytes per weight
  using R = Ring<FP8, TOK>;
  constexpr int NJ = Cols<TOK>::kMmas, TPG = Cols<TOK>::kTpg;
  constexpr int Q = R::kPieces, KE = 64 / EB;  // K elements of 64 bytes of weights
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tq = lane & 3;  // MMA fragment row / column, K group
  const int tok = g / TPG;                 // token of this lane's column
  const bool first_lane = lane % (4 * TPG) == 0;
  const int T = p.T, H = p.H, E = p.E, I = p.I, k = p.k;
  if (tid < kMaxExperts) sm.used[tid] = 0;
  // what does not depend on the routing is worked out before the wait
  const int n0 = (int)((int64_t)blockIdx.x * H / gridDim.x);
  const int n1 = (int)((int64_t)(blockIdx.x + 1) * H / gridDim.x);
  const uint32_t rb1 = (uint32_t)H * EB, rb2 = (uint32_t)I * EB;  // bytes of a weight row
  const int S1 = (int)((rb1 + 127) >> 7), S2 = (int)((rb2 + 127) >> 7);  // 128-byte steps of a row
  const int kb1 = (int)(rb1 >> 6), kb2 = (int)(rb2 >> 6);                // 64-byte K blocks
  const int P1 = (H + 127) >> 7;                                         // powers of two of a row of x
  const int tiles_e = I >> 3;                                            // FC1 row tiles of an expert
  const unsigned magic = 0xffffffffu / (unsigned)tiles_e;
  static_assert(R::kDepth <= kMaxDepth && kMaxExperts <= kThreadsL, "shared tables");
  if (tid < kWarps) {
    for (int i = 0; i < R::kDepth; ++i) {
      ptx::mbar_init(&sm.full[tid][i], 32);
      ptx::mbar_init(&sm.empty[tid][i], 1);
    }
    ptx::fence_mbar_init();
  }
  if (tid == 0) {
    sm.published = 1;
    sm.fc1_done = sm.abort = 0;
  }
  __syncthreads();
  pdl_wait();

  // ---- routing (every CTA by itself; warp t: token t)
  int first_claim = 0;
  if (tid == 2 * kThreadsL - 1) first_claim = atomicAdd(&p.ctr[0], 2);
  // More than 64 experts of few tokens: the logits by all warps, 32 experts at a time,
  // if each warp has one such part at most (one token, 256 experts: 58.2 us against
  // 60.6 by the token's warp alone; eight tokens, four parts a warp, 200.2 against
  // 199.4, and with 64 experts 0.2 us more).
  const unsigned* keys = nullptr;
  const int parts = (E + 31) >> 5;
  if (!p.ids_in && E > 64 && T * parts <= 2 * kWarps) {
    unsigned* all = reinterpret_cast<unsigned*>(red);  // [T][E]
    static_assert(sizeof(red) >= sizeof(unsigned) * kLayerMaxT * kMaxExperts, "keys");
    if (warp < T * parts) {
      const int t = warp / parts;
      layer_part(p.logits ? p.logits + (size_t)t * E : nullptr, p.part + (size_t)t * E, p.bias, p.ssq + t, T * E, E, H,
                 p.eps, warp - t * parts, all + t * E, &sm.r[t]);
    }
    __syncthreads();
    keys = all + warp * E;
  }
  if (warp < T) {
    const float ss = lane < kLayerChunks ? __ldcg(&p.ssq[lane * kLayerMaxT + warp]) : 0.f;
    if (p.ids_in) {
      if (lane < k) {
        sm.ids[warp][lane] = p.ids_in[warp * k + lane];
        sm.w[warp][lane] = p.tw_in[warp * k + lane];
      }
      const float r = 1.0f / sqrtf(warp_sum(ss) / (float)H + p.eps);
      if (lane == 0) sm.r[warp] = r;
    } else if (E <= 32) {
      layer_topk<1>(p, warp, lane, ss, keys, &sm);
    } else if (E <= 64) {
      layer_topk<2>(p, warp, lane, ss, keys, &sm);
    } else if (E <= 128) {
      layer_topk<4>(p, warp, lane, ss, keys, &sm);
    } else {
      layer_topk<8>(p, warp, lane, ss, keys, &sm);
    }
    // the token's experts: lane j, its j-th
    __syncwarp();
    const int id = lane < k ? sm.ids[warp][lane] : -1;
    if (id >= 0 && id < E) atomicOr(&sm.used[id], 1u << warp);
    if (blockIdx.x == 0 && lane < k) {
      if (p.ids_out) p.ids_out[warp * k + lane] = id;
      if (p.tw_out) p.tw_out[warp * k + lane] = sm.w[warp][lane];
      if (id < 0 || id >= E) flag_status(p.status, MOE_ERR_INVALID_ARG);
    }
  }
  if (tid == 2 * kThreadsL - 1) {
    sm.claim[0] = first_claim;
    sm.claim[1] = first_claim + 1;
  }
  __syncthreads();
  // active experts in ascending order (thread e: expert e; E <= 256)
  {
    const unsigned mask = tid < kMaxExperts ? sm.used[tid] : 0u;
    const unsigned act = __ballot_sync(0xffffffffu, mask != 0);
    if (lane == 0 && warp < kWarps) sm.warp_cnt[warp] = __popc(act);
    __syncthreads();
    if (mask) {
      int at = __popc(act & ((1u << lane) - 1));
      for (int w = 0; w < warp; ++w) at += sm.warp_cnt[w];
      sm.expert[at] = tid;
      sm.mask[at] = mask;
      sm.slot[tid] = at;
      *reinterpret_cast<int4*>(&sm.pair[at][0]) = make_int4(-1, -1, -1, -1);
      *reinterpret_cast<int4*>(&sm.pair[at][4]) = make_int4(-1, -1, -1, -1);
    }
    __syncthreads();
    if (warp < T && lane < k) {
      const int id = sm.ids[warp][lane];
      if (id >= 0 && id < E) {
        // an expert given twice counts once, with the sum of its weights
        bool first = true;
        float w = 0.f;
        for (int j = 0; j < k; ++j)
          if (sm.ids[warp][j] == id) {
            if (j < lane) first = false;
            w += sm.w[warp][j];
          }
        if (first) {
          sm.pair[sm.slot[id]][warp] = warp * k + lane;
          sm.wt[sm.slot[id]][warp] = w;
        }
      }
    }
    __syncthreads();
  }
  int n_act = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) n_act += sm.warp_cnt[w];

  // ---- work.  FC1 row tiles (8 gate + 8 up rows) in claims of two, the last
  // ones (one per CTA) single, the K steps of a claim interleaved over the
  // warps.  FC2: output rows [n0, n1) in units of 32, all experts' K
  // steps in one sequence of which warp w takes the w-th eighth.
  const int tiles = n_act * tiles_e;
  const int singles = min(tiles, (int)gridDim.x & ~1);
  const int pairs = (tiles - singles) >> 1;  // tiles and singles are even
  const int claims = pairs + singles;
  // expert slot and first intermediate column of a claim
  auto claim_at = [&](int c, int& a, int& i0) {
    const int tile = c < pairs ? 2 * c : c + pairs;
    a = (int)__umulhi((unsigned)tile, magic);  // tile / tiles_e, or one less
    int rest = tile - a * tiles_e;
    if (rest >= tiles_e) {
      ++a;
      rest -= tiles_e;
    }
    i0 = rest * 8;
  };

  const int wk = warp % kWarps;  // consumer whose steps these are
  const int q0 = n_act * S2 * wk / kWarps, q1 = n_act * S2 * (wk + 1) / kWarps;  // FC2 steps of a unit
  const int a_first = n_act * wk / kWarps, s_first = q0 - a_first * S2;  // (q0 / S2)
  const int units = (n1 - n0 + 31) / 32;
  unsigned char* ring = ring_all + wk * R::kWarp;
  const size_t x_term = (size_t)T * H, a_term = (size_t)T * k * I;  // elements of a term

  if (warp >= kWarps) {
    // -------------------------------------------------------------- producer --
    const uint32_t ring_u = ptx::smem_u32(ring);
    // block scales: one row of the scale matrix per 128 weight rows, one column
    // per K step; channel scales: one per row
    const int rs = p.block_scales ? 7 : 0, ks = p.block_scales ? 1 : 0;
    const int kg1 = p.block_scales ? H >> 7 : 1, kg2 = p.block_scales ? I >> 7 : 1;
    int slot = 0;
    uint32_t ph = 1;  // the ring starts empty
    // Weights of a step: this lane's first row at the step, to the second tile and
    // to a tile's lower 8 rows (bytes), bit 2 * tile + half of `ok` where the lane's
    // row is wanted.  `two`: the step's second K block exists (else zeros).
    auto copy_a = [&](int sl, const unsigned char* src, uint32_t ts, uint32_t hs, unsigned ok, bool two) {
      const uint32_t dst = ring_u + sl * R::kStage + lane * 16;
      const unsigned char *s1 = src + hs, *s2 = src + ts, *s3 = s2 + hs;
      if (ok == 15u && two) {
        cp_async16(dst, src);
        cp_async16(dst + 512, src + 64);
        cp_async16(dst + 2 * 512, s1);
        cp_async16(dst + 3 * 512, s1 + 64);
        cp_async16(dst + 4 * 512, s2);
        cp_async16(dst + 5 * 512, s2 + 64);
        cp_async16(dst + 6 * 512, s3);
        cp_async16(dst + 7 * 512, s3 + 64);
      } else {
        const unsigned char* r[4] = {src, s1, s2, s3};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((ok >> i) & 1u) {
            cp_async16(dst + 1024 * i, r[i]);
            cp_async16z(dst + 1024 * i + 512, two ? r[i] + 64 : r[i], two ? 16 : 0);
          }
        }
      }
    };
    // This lane's column of the activations at the step, to the next MMA's column.
    auto copy_b = [&](int sl, const uint16_t* b, size_t bj, bool two) {
      const uint32_t dst = ring_u + sl * R::kStage + kStepA + lane * 16;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          cp_async16_l1(dst + (j * Q + q) * 512, b + j * bj + q * 8, 16);
          cp_async16_l1(dst + ((NJ + j) * Q + q) * 512, b + j * bj + (two ? KE : 0) + q * 8, two ? 16 : 0);
        }
      }
    };
    auto wait_empty = [&]() -> bool { return ptx::mbar_wait(&sm.empty[wk][slot], ph, &sm.abort); };
    auto next_slot = [&]() {
      if (++slot == R::kDepth) {
        slot = 0;
        ph ^= 1;
      }
    };
    // Waits until *flag >= want (a word of shared memory that a consumer writes).
    auto wait_flag = [&](int* flag, int want) -> bool {
      const long long t0 = clock64();
      while (*(volatile int*)flag < want) {
        if (*(volatile int*)&sm.abort) return false;
        if (clock64() - t0 > ptx::kSpinLimitCycles) {
          *(volatile int*)&sm.abort = 1;
          return false;
        }
        __nanosleep(64);
      }
      __threadfence_block();
      return true;
    };
    bool ok = true;
    // FC1 (a warp beyond the steps of a row has none)
    for (int n = 0; ok && wk < S1; ++n) {
      if (!(ok = wait_flag(&sm.published, n))) break;
      const int c = *(volatile int*)&sm.claim[n & 3];
      if (c >= claims) break;
      int a, i0;
      claim_at(c, a, i0);
      const int e = sm.expert[a];
      const unsigned char* src =
          static_cast<const unsigned char*>(p.w13) + ((size_t)e * 2 * I + i0 + g) * rb1 + wk * 128 + tq * 16;
      const bool on = (sm.mask[a] >> tok) & 1u;
      const uint16_t* b =
          p.xt + (size_t)(g % TPG) * x_term + (size_t)(on ? tok : 0) * H + wk * 2 * KE + tq * 8 * Q;
      const float *sc = nullptr, *pw = nullptr;
      bool sok = false;
      if constexpr (FP8) {
        const int row = i0 + (lane & 7) + ((lane & 8) ? I : 0) + ((lane & 16) ? 8 : 0);
        sok = c < pairs || lane < 16;
        sc = p.s13 + ((size_t)e * (2 * I >> rs) + ((sok ? row : 0) >> rs)) * kg1 + wk * ks;
        pw = p.xpow + (on ? tok : 0) * P1 + wk;
      }
#pragma unroll 1
      for (int step = wk; step < S1; step += kWarps) {
        if (!(ok = wait_empty())) break;
        const bool two = !FP8 || 2 * step + 1 < kb1;
        copy_a(slot, src, 8 * rb1, (uint32_t)I * rb1, c < pairs ? 15u : 3u, two);
        if (on) {
          copy_b(slot, b, TPG * x_term, two);
          if (FP8 && first_lane) cp_async4(ring_u + slot * R::kStage + R::kPowAt + tok * 4, pw);
        }
        if (FP8 && sok) cp_async4(ring_u + slot * R::kStage + R::kScaleAt + lane * 4, sc);
        cp_arrive(&sm.full[wk][slot]);
        next_slot();
        src += kWarps * 128;
        b += kWarps * 2 * KE;
        if constexpr (FP8) {
          sc += kWarps * ks;
          pw += kWarps;
        }
      }
    }
    // FC2: (unit, expert, step) in order; the first steps' weights are copied
    // before the intermediate is there
    struct At {
      int u, a, s;
    };
    const int total = (q1 - q0) * units;
    auto advance = [&](At& t) {
      if (t.a * S2 + ++t.s == q1) {
        ++t.u;
        t.a = a_first;
        t.s = s_first;
      } else if (t.s == S2) {
        ++t.a;
        t.s = 0;
      }
    };
    auto step_a = [&](int sl, const At& t) {
      const int row0 = n0 + 32 * t.u, e = sm.expert[t.a];
      unsigned want = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) want |= (row0 + g + 8 * i < n1 ? 1u : 0u) << i;
      copy_a(sl, static_cast<const unsigned char*>(p.w2) + ((size_t)e * H + row0 + g) * rb2 + t.s * 128 + tq * 16,
             16 * rb2, 8 * rb2, want, !FP8 || 2 * t.s + 1 < kb2);
      if (FP8 && row0 + lane < n1)
        cp_async4(ring_u + sl * R::kStage + R::kScaleAt + lane * 4,
                  p.s2 + ((size_t)e * (H >> rs) + ((row0 + lane) >> rs)) * kg2 + t.s * ks);
    };
    auto step_b = [&](int sl, const At& t) {
      const int pr = sm.pair[t.a][tok];
      if (pr >= 0) {
        const bool two = !FP8 || 2 * t.s + 1 < kb2;
        copy_b(sl, p.at + (size_t)(g % TPG) * a_term + (size_t)pr * I + t.s * 2 * KE + tq * 8 * Q, TPG * a_term, two);
        // lane tq of the token's first column: the eight groups of K block tq (an
        // absent block's exponents are 0, its factors too)
        if (FP8 && g % TPG == 0 && tq < 2) {
          const bool there = two || tq == 0;
          cp_async8(ring_u + sl * R::kStage + R::kPowAt + (tq * TOK + tok) * 8,
                    p.apow + (size_t)pr * (I >> 3) + t.s * 16 + (there ? tq * 8 : 0), there ? 8 : 0);
        }
      }
    };
    if (ok && total > 0) {
      const int early = min(R::kDepth, total);
      const int slot0 = slot;
      const uint32_t ph0 = ph;
      At ta{0, a_first, s_first}, tb = ta;
      for (int i = 0; ok && i < early; ++i) {
        if (!(ok = wait_empty())) break;
        step_a(slot, ta);
        next_slot();
        advance(ta);
      }
      if (ok) ok = wait_flag(&sm.fc1_done, 1);
      slot = slot0;
      ph = ph0;
#pragma unroll 1
      for (int i = 0; ok && i < total; ++i) {
        if (i >= early) {
          if (!(ok = wait_empty())) break;
          step_a(slot, tb);
        }
        step_b(slot, tb);
        cp_arrive(&sm.full[wk][slot]);
        next_slot();
        advance(tb);
      }
    }
    cp_wait_all();
    return -1;
  }

  // ---------------------------------------------------------------- consumers --
  // One step: acc[MMA][tile] += weights of the step * the columns.  What was not
  // copied (rows that are not wanted, tokens that do not use the expert) is
  // whatever the ring held: it only reaches sums that are not used.  FP8: s, the
  // scales of the lane's rows times the powers of two of its two columns.
  using Sums = float[NJ][2][4];
  constexpr int NC = TPG > 1 ? 1 : 2;  // tokens of the lane's two columns
  int slot = 0;
  uint32_t ph = 0;
  bool arrived = true;
  // FC2 with FP8: the 8-column groups of the lane's column are brought to the
  // largest exponent among the step's sixteen.
  auto multiply = [&](bool fc2, Sums& acc, float (&s)[4][NC]) {
    arrived = ptx::mbar_wait(&sm.full[warp][slot], ph, &sm.abort) && arrived;
    const unsigned char* st = ring + slot * R::kStage;
    const uint4* sp = reinterpret_cast<const uint4*>(st) + lane;
    int top = 0;
    if (FP8 && fc2) {
      const uint2 e0 = *reinterpret_cast<const uint2*>(st + R::kPowAt + tok * 8);
      const uint2 e1 = *reinterpret_cast<const uint2*>(st + R::kPowAt + (TOK + tok) * 8);
      constexpr unsigned kEven = 0x00ff00ffu;  // of the largest 16-bit word, the upper byte is the largest upper byte
      const unsigned odd = __vmaxu2(__vmaxu2(e0.x, e0.y), __vmaxu2(e1.x, e1.y));
      const unsigned even = __vmaxu2(__vmaxu2(e0.x & kEven, e0.y & kEven), __vmaxu2(e1.x & kEven, e1.y & kEven));
      const unsigned m = __vmaxu2((odd >> 8) & kEven, even);
      top = (int)max(m & 0xffffu, m >> 16);
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      uint4 b[NJ][Q];
#pragma unroll
      for (int j = 0; j < NJ * Q; ++j) b[j / Q][j % Q] = sp[kStepA / 16 + (kb * NJ * Q + j) * 32];
      if (FP8 && fc2) {
        const unsigned ex = *reinterpret_cast<const uint16_t*>(st + R::kPowAt + (kb * TOK + tok) * 8 + tq * 2);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int d = (int)((ex >> (8 * q)) & 255u) - top;  // <= 0: a power of two (0 below 2^-24)
          const __half2 f = __float2half2_rn(__uint_as_float((uint32_t)max(127 + d, 0) << 23));
#pragma unroll
          for (int j = 0; j < NJ; ++j) b[j][q] = hmul2x4(b[j][q], *reinterpret_cast<const uint32_t*>(&f));
        }
      }
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        const uint4 lo = sp[((tl * 2 + 0) * 2 + kb) * 32], hi = sp[((tl * 2 + 1) * 2 + kb) * 32];  // rows g, g + 8
        if constexpr (FP8) {
          const uint32_t c0[4] = {lo.x, lo.y, lo.z, lo.w}, c1[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_f16(c0[m], a0, a2);
            e4m3x4_f16(c1[m], a1, a3);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const uint4 v = b[j][(m >> 1) % Q];
              mma_16816<true>(acc[j][tl], a0, a1, a2, a3, (m & 1) ? v.z : v.x, (m & 1) ? v.w : v.y);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            mma_16816<false>(acc[j][tl], lo.x, hi.x, lo.y, hi.y, b[j][0].x, b[j][0].y);
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            mma_16816<false>(acc[j][tl], lo.z, hi.z, lo.w, hi.w, b[j][0].z, b[j][0].w);
        }
      }
    }
    if constexpr (FP8) {
      const float* pw = reinterpret_cast<const float*>(st + R::kPowAt) + 2 * tq / TPG;
      const float mine = pow_down(top);
      float down[NC];  // powers of two of the lane's columns
#pragma unroll
      for (int c = 0; c < NC; ++c)  // (lane 4 TPG t holds that of token t)
        down[c] = fc2 ? __shfl_sync(0xffffffffu, mine, (2 * tq / TPG + c) * 4 * TPG) : pw[c];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = *reinterpret_cast<const float*>(st + R::kScaleAt + (g + 8 * i) * 4);
#pragma unroll
        for (int c = 0; c < NC; ++c) s[i][c] = w * down[c];
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sm.empty[warp][slot]);
    if (++slot == R::kDepth) {
      slot = 0;
      ph ^= 1;
    }
  };
  // tot += s * acc for the tokens in `mask` (bit i: token i); acc = 0.  A token
  // outside the mask gets nothing (not 0 times a weight that may not be finite).
  auto fold = [&](Sums& tot, Sums& acc, const float (&s)[4][NC], unsigned mask) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if ((mask >> (2 * tq / TPG + c)) & 1u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (NC == 2 && (i & 1) != c) continue;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int tl = 0; tl < 2; ++tl)
              tot[j][tl][i] = FP8 ? fmaf(s[tl * 2 + (i >> 1)][c], acc[j][tl][i], tot[j][tl][i])
                                  : tot[j][tl][i] + acc[j][tl][i];
        }
      }
#pragma unroll
    for (int i = 0; i < NJ * 8; ++i) acc[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
  };
  // This warp's partial sums, the terms of a token added, into rd [2 tiles][16
  // rows][8 tokens]; tot = 0.
  auto store_red = [&](float* rd, Sums& tot) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // rows g and g + 8
        float* d = rd + (tl * 16 + 8 * h + g) * 8;
        if (TPG == 2) d[tq] = tot[0][tl][2 * h] + tot[0][tl][2 * h + 1];
        else
          *reinterpret_cast<float2*>(d + 2 * tq) =
              make_float2(tot[0][tl][2 * h] + tot[NJ - 1][tl][2 * h], tot[0][tl][2 * h + 1] + tot[NJ - 1][tl][2 * h + 1]);
      }
#pragma unroll
    for (int i = 0; i < NJ * 8; ++i) tot[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
  };
  // Thread 0 waits until *ctr >= want; false (for all) when the wait runs out.
  auto wait_for = [&](const int* ctr, int want) -> bool {
    if (tid == 0) {
      const long long t0 = clock64();
      int seen;
      do {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(ctr) : "memory");
      } while (seen < want && clock64() - t0 < ptx::kSpinLimitCycles);
      sm.in_time = seen >= want;
      if (seen < want) *(volatile int*)&sm.abort = 1;
      __threadfence();
    }
    consumer_sync();
    return sm.in_time != 0;
  };

  int buf = 0, my_tiles = 0;
  float sc[4][NC] = {};
  Sums acc = {}, tot = {};

  // ---- FC1
  for (int n = 0;; ++n) {
    const int c = sm.claim[n & 3];
    if (c >= claims) break;
    int next_claim = claims;
    if (tid == 0) next_claim = atomicAdd(&p.ctr[0], 1);  // used two claims from here
    int a, i0;
    claim_at(c, a, i0);
    const unsigned mask = sm.mask[a];
    const bool second = c < pairs;
#pragma unroll 1
    for (int step = warp; step < S1; step += kWarps) {
      multiply(false, acc, sc);
      if constexpr (FP8) fold(tot, acc, sc, mask);
    }
    if constexpr (!FP8) fold(tot, acc, sc, mask);
    store_red(red[buf] + warp * 256, tot);
    if (tid == 0) {
      sm.claim[(n + 2) & 3] = next_claim;
      __threadfence_block();
      *(volatile int*)&sm.published = n + 2;
    }
    consumer_sync();
    // the claim's 16 intermediate columns: warp t, token t; each half warp adds the
    // partial sums of four warps
    if ((mask >> warp) & 1u) {
      const int il = lane & 15;
      const float* s = red[buf] + ((il >> 3) * 16 + (il & 7)) * 8 + warp + (lane >> 4) * 1024;
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        gate += s[w * 256];
        up += s[w * 256 + 64];
      }
      gate += __shfl_xor_sync(0xffffffffu, gate, 16);
      up += __shfl_xor_sync(0xffffffffu, up, 16);
      const float r = sm.r[warp];
      // the routing weight goes into the intermediate, so FC2 adds the token's
      // experts without a factor
      float v = silu_f(gate * r) * (up * r) * sm.wt[a][warp];
      const bool mine = lane < (second ? 16 : 8);
      const int pr = sm.pair[a][warp];
      if constexpr (FP8) {  // eight columns share a power of two
        float m = fabsf(v);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int ex = pow_exponent(m);
        v *= pow_up(ex);
        if (mine && (il & 7) == 0) p.apow[(size_t)pr * (I >> 3) + (i0 + il) / 8] = (uint8_t)ex;
      }
      if (mine) {
        const size_t at = (size_t)pr * I + i0 + il;
        split16<FP8>(v, p.at[at], p.at[at + a_term]);
      }
    }
    my_tiles += second ? 2 : 1;
    buf ^= 1;
  }
  // ---- all FC1 tiles done (this CTA's are counted once its writes are there)
  consumer_sync();
  if (tid == 0 && my_tiles) {
    __threadfence();
    atomicAdd(&p.ctr[1], my_tiles);
  }
  if (!wait_for(p.ctr + 1, tiles)) {
    if (tid == 0) flag_status(p.status, MOE_ERR_TIMEOUT);
    return -1;
  }
  if (tid == 0) {
    __threadfence_block();
    *(volatile int*)&sm.fc1_done = 1;
  }

  // ---- FC2: this CTA's output rows over all active experts
  for (int u = 0; u < units; ++u) {
    int a = a_first, s_at = s_first;
    for (int q = q0; q < q1;) {
      const unsigned mask = sm.mask[a];
      const int end = min(q1, q + S2 - s_at);
#pragma unroll 1
      for (; q < end; ++q) {
        multiply(true, acc, sc);
        if constexpr (FP8) fold(tot, acc, sc, mask);
      }
      if constexpr (!FP8) fold(tot, acc, sc, mask);
      ++a;
      s_at = 0;
    }
    store_red(red[buf] + warp * 256, tot);
    consumer_sync();
    const int row = n0 + 32 * u + lane, t = warp;
    if (t < T && row < n1) {
      const float* s = red[buf] + lane * 8 + t;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s[w * 256];
      const size_t at = (size_t)t * H + row;
      if (has_tail) p.f[at] = v;
      else static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(v);
    }
    buf ^= 1;
  }
  if (!arrived) flag_status(p.status, MOE_ERR_TIMEOUT);
  if (!has_tail) return -1;

  // ---- tail: the last T CTAs to finish take a row each.  (When they wait for
  // one another, fewer than T CTAs are unfinished, and the others have left their
  // SMs to them.)
  consumer_sync();
  if (tid == 0) {
    __threadfence();
    sm.flag = atomicAdd(&p.ctr[2], 1) - ((int)gridDim.x - T);
  }
  consumer_sync();
  return sm.flag;
}

// An SM does a tail row only every 152 / T calls, and by then the code of the tail has
// left its instruction cache, and L2 as well (weights went through it): fetching it
// again cost 1 us of 62 (one token) and more.  So one warp of every CTA runs it once
// without effect while the others already wait for the first launch.  (Not with E4M3
// weights and eight token columns: that kernel has no register to spare, and with the
// loop around it its steps spill: eight tokens 168 us against 153.)  It reads and writes
// shared memory that holds nothing yet (its own columns of `f` and one word of sm.sum, before
// the ring's first copies): no result depends on it.
template <bool FP8, int TOK>
__global__ void __launch_bounds__(2 * kThreadsL, 1) layer_experts_kernel(const LayerP p, const TailP tail,
                                                                     int has_tail) {
  using R = Ring<FP8, TOK>;
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ LayerSmem sm;
  __shared__ __align__(16) float red[2][kRed];
  const int tid = threadIdx.x, H = p.H;
  pdl_trigger();
  const bool staged = (size_t)H * 16 <= (size_t)R::kBytes;
  static_assert(kLayerMaxH * 4 <= R::kBytes, "f fits in any case");
  bool dry = !(FP8 && TOK == 8) && has_tail && staged && tid / 32 == kWarps - 1;
  int t = 0, grow = 0;
  float factor = 0.f;
#pragma unroll 1
  for (;;) {  // (one copy of the tail's code, run twice)
    if (!dry) {
      t = layer_experts<FP8, TOK>(p, has_tail, ring_all, sm, red);
      if (t < 0) return;
      grow = tail_gate_row(tail, t, tid == 0 ? p.status : nullptr);
      factor = tail_row_factor(tail, grow);
      // the row's inputs into the ring's shared memory: f [H] fp32, residual, gate
      // row (room for fp32 each), the norms' weights
      auto stage = [&](size_t at, const void* src, size_t bytes) {
        if (src)
#pragma unroll 1
          for (size_t o = tid * 16; o < bytes; o += kThreadsL * 16)
            cp_async16(ptx::smem_u32(ring_all + at + o), static_cast<const unsigned char*>(src) + o);
      };
      if (staged) {
        const size_t res_b = (size_t)H * (tail.res_f32 ? 4 : 2), gate_b = (size_t)H * (tail.gate_f32 ? 4 : 2);
        if (tail.residual) stage((size_t)H * 4, static_cast<const unsigned char*>(tail.residual) + t * res_b, res_b);
        if (tail.gate && tail.gate_cols != 1 && grow >= 0)
          stage((size_t)H * 8, static_cast<const unsigned char*>(tail.gate) + grow * gate_b, gate_b);
        stage((size_t)H * 12, tail.post_w, (size_t)H * 2);
        stage((size_t)H * 14, tail.next_w, (size_t)H * 2);
      }
      if (tid == 0) {
        const long long t0 = clock64();
        int seen;
        do {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(p.ctr + 2) : "memory");
        } while (seen < (int)gridDim.x && clock64() - t0 < ptx::kSpinLimitCycles);
        if (seen < (int)gridDim.x) flag_status(p.status, MOE_ERR_TIMEOUT);
        __threadfence();
      }
      consumer_sync();
      stage(0, p.f + (size_t)t * H, (size_t)H * 4);
      cp_wait_all();
    }
    layer_tail_row(p, tail, t, grow, factor, ring_all, staged, sm.sum, dry);
    if (!dry) return;
    dry = false;
  }
}

struct LayerWs {
  size_t xt, at, xpow, apow, ssq, part, f, ctr, total;
};

LayerWs layer_layout(int T, int H, int E, int I, int k, bool fp8) {
  LayerWs w{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~(size_t)255;
    return at;
  };
  const size_t t = T > 0 ? T : 1;
  w.xt = take(t * H * 4);
  w.at = take(t * k * I * 4);
  w.xpow = take(fp8 ? t * ((H + 127) / 128) * 4 : 0);
  w.apow = take(fp8 ? t * k * (I / 8) : 0);
  w.ssq = take((size_t)kLayerChunks * kLayerMaxT * 4);
  w.part = take((size_t)kLayerChunks * t * E * 4);
  w.f = take(t * H * 4);
  w.ctr = take(kCtrInts * 4);
  w.total = o;
  return w;
}

}  // namespace

size_t layer_workspace_bytes(int T, int H, int E, int I, int k, bool fp8) {
  return layer_layout(T, H, E, I, k, fp8).total;
}

cudaError_t launch_layer(const LayerArgs& a, const TailP* tail, int sms, int* status, cudaStream_t st) {
  const LayerWs w = layer_layout(a.T, a.H, a.E, a.I, a.k, a.fp8);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  LayerP p{};
  p.x = static_cast<const bf16*>(a.x);
  p.norm_w = static_cast<const bf16*>(a.norm_w);
  p.router_w = a.router_w;
  p.logits = a.logits;
  p.bias = a.bias;
  p.ids_in = a.ids_in;
  p.tw_in = a.tw_in;
  p.w13 = a.w13;
  p.w2 = a.w2;
  p.s13 = a.s13;
  p.s2 = a.s2;
  p.ids_out = a.ids_out;
  p.tw_out = a.tw_out;
  p.out = a.out;
  p.T = a.T;
  p.H = a.H;
  p.E = a.E;
  p.I = a.I;
  p.k = a.k;
  p.block_scales = a.block_scales;
  p.eps = a.eps;
  p.xt = reinterpret_cast<uint16_t*>(ws + w.xt);
  p.at = reinterpret_cast<uint16_t*>(ws + w.at);
  p.xpow = reinterpret_cast<float*>(ws + w.xpow);
  p.apow = ws + w.apow;
  p.ssq = reinterpret_cast<float*>(ws + w.ssq);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.f = reinterpret_cast<float*>(ws + w.f);
  p.ctr = reinterpret_cast<int*>(ws + w.ctr);
  p.status = status;
  int rows = 0;  // of the largest chunk
  for (int c = 0; c < kLayerChunks; ++c) {
    const Chunk ch = layer_chunk(a.H, c);
    if (ch.k1 - ch.k0 > rows) rows = ch.k1 - ch.k0;
  }
  const int tt = a.T <= 2 ? 2 : (a.T <= 4 ? 4 : kLayerMaxT);
  const int route_smem = a.router_w ? rows * tt * 4 : 0;  // up to 32 KB beside the static part
  auto route = a.fp8 ? layer_route_kernel<true, kLayerMaxT> : layer_route_kernel<false, kLayerMaxT>;
  if (tt == 2) route = a.fp8 ? layer_route_kernel<true, 2> : layer_route_kernel<false, 2>;
  if (tt == 4) route = a.fp8 ? layer_route_kernel<true, 4> : layer_route_kernel<false, 4>;
  cudaError_t e = cudaSuccess;
  if (route_smem > (24 << 10))  // (one limit for all calls: other threads may launch between)
    e = cudaFuncSetAttribute(route, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kLayerMaxH / kLayerChunks * kLayerMaxT * 4);
  if (e != cudaSuccess) return e;
  e = launch_kernel(route, dim3(kLayerChunks, a.router_w ? (a.E + 31) / 32 : 1), dim3(32 * kRouteWarps),
                    (size_t)route_smem, st, p);
  if (e != cudaSuccess) return e;
  auto kern = layer_experts_kernel<false, 8>;
  int smem = Ring<false, 8>::kBytes;
#define MOE_LAYER_KERNEL(F, TOK)          \
  {                                       \
    kern = layer_experts_kernel<F, TOK>;  \
    smem = Ring<F, TOK>::kBytes;          \
  }
  if (a.fp8) {
    if (a.T <= 4) MOE_LAYER_KERNEL(true, 4)
    else MOE_LAYER_KERNEL(true, 8)
  } else if (a.T <= 4) {
    MOE_LAYER_KERNEL(false, 4)
  }
#undef MOE_LAYER_KERNEL
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(sms), dim3(2 * kThreadsL), smem, st, p, tail ? *tail : TailP{},
                       tail ? 1 : 0);
}

}  // namespace moe
