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
// Products: the weights are the 16 x 16 operand of m16n8k16 MMAs, the (at most
// 8) tokens the 8 columns; fp32 accumulation.  Activations enter as two 16-bit
// terms hi + lo, so neither x_hat nor the intermediate is rounded to 16 bits:
// bf16 terms for bf16 weights (16 bits of mantissa); fp16 terms for E4M3 weights
// (22 bits), because E4M3 -> fp16 is one instruction for two weights and
// E4M3 -> bf16 four.  fp16 has little range, so its terms carry a power of two:
// one per token and K chunk for x (the chunk's maximum), one per 8 columns for
// the intermediate (a row tile's), brought to the pair's largest by an exact
// fp16 product when they are used.
//
// A warp reads its own operands: each lane copies exactly the 16-byte pieces it
// will feed to its MMAs into its own part of shared memory (cp.async, a few
// steps ahead) and reads them back, so the stream needs no barrier, and the
// first W2 pieces are already on their way while the CTA waits for the other
// CTAs' FC1 tiles.  The order of the K elements inside a piece is the same for
// both operands and therefore free.  The activations go the same way as the
// weights: a plain load of them would wait behind the copies in flight (4 us of
// them with 160 KB per SM).
//
// mma.sync and not tcgen05: at 8 columns the tensor work is 1/16 of what the
// legacy instruction sustains at this memory rate, a fragment load straight from
// the copied bytes needs no descriptor layout, and accumulators in registers
// spare the TMEM round trip between short row tiles.
#include "block_tail.cuh"
#include "kernels.h"
#include "tail.h"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsL = 32 * kWarps;

// Per-warp stage of the copy ring: weights [2 tiles][2 row halves][2 K blocks]
// [32 lanes] of 16 bytes; activations [2 K blocks][hi, lo][pieces][TOK tokens]
// [4 lanes] of 16 bytes; FP8: the scales of the 32 rows and [2 K blocks][8
// tokens][8 groups] exponents.  TOK is 4 where T <= 4: the room goes to more
// steps in flight.
constexpr int kStepA = 4096;
template <bool FP8, int TOK>
struct Ring {
  static constexpr int kPieceB = TOK * 64;
  static constexpr int kScaleAt = kStepA + 4 * (FP8 ? 2 : 1) * kPieceB;  // scales of the 32 rows
  static constexpr int kPowAt = kScaleAt + 128;  // exponents of the intermediate's 8-column groups
  static constexpr int kStage = kScaleAt + (FP8 ? 128 + 128 : 0);
  static constexpr int kDepth = (200 << 10) / (kWarps * kStage);  // 3 .. 5 steps
  static constexpr int kWarp = kDepth * kStage;
  static constexpr int kBytes = kWarps * kWarp;
  // Groups of warps that take FC1 claims of their own.
  static constexpr int kGroups = 1;
};
constexpr int kGroupRed = 2 * 2 * 16 * 8;  // floats: two buffers of two row tiles, per warp of the group
constexpr int kMaxPairs = kLayerMaxT * kMaxTopK;
constexpr int kCtrPow = 8;  // ctr: largest exponent of each pair's intermediate
constexpr int kCtrInts = kCtrPow + kMaxPairs;

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
  uint16_t *hi, *lo;          // x w [T, H] in two terms (bf16, or fp16 with FP8 weights)
  uint16_t *act_hi, *act_lo;  // intermediate [T k, I], times the routing weight
  uint8_t* act_pow;           // FP8: its exponents (pow_exponent) [T k, I / 8]
  float *ssq, *xpow;          // sums of squares and factors of x w [chunks, 8]
  float *part, *f;            // partial logits [chunks, T, E], f [T, H]
  int* ctr;                   // [0] FC1 claims, [1] FC1 tiles done, [2] CTAs finished, [8..] kCtrPow
  int* status;
};

// K chunk c covers the units [c n / 16, (c + 1) n / 16) of 128 columns (the last
// unit may be 64 wide), so that a 128-column step of the FP8 products lies in one.
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
// Grid (kLayerChunks, groups of 32 experts): K chunk c, experts 32y .. 32y+31.
// Latency is all there is: each warp has its rows of W_r (16 at H = 4096) on
// their way before it waits for anything.
constexpr int kRouteWarps = 16;

template <bool F16>
__global__ void __launch_bounds__(32 * kRouteWarps) layer_route_kernel(const LayerP p) {
  extern __shared__ __align__(16) float xw[];  // [rows of the chunk][8 tokens]
  __shared__ float red[kRouteWarps][kLayerMaxT][32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x;
  const Chunk ch = layer_chunk(p.H, c);
  const int k0 = ch.k0, rows = ch.k1 - ch.k0;
  if (c == 0 && blockIdx.y == 0 && tid < kCtrInts) p.ctr[tid] = 0;
  const int e = blockIdx.y * 32 + lane;
  const float* wr = p.router_w ? p.router_w + (size_t)k0 * p.E + e : nullptr;
  constexpr int U = 16;
  float wv[U];
  if (wr) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = warp + kRouteWarps * u;
      wv[u] = (r < rows && e < p.E) ? wr[(size_t)r * p.E] : 0.f;
    }
  }
  // warp t: token t (zeros beyond the last)
  if (warp < kLayerMaxT) {
    const size_t row = (size_t)(warp < p.T ? warp : 0) * p.H + k0;
    float ss = 0.f, up = 1.f;
    if (F16 && warp < p.T) {  // the chunk's power of two
      float m = 0.f;
      for (int v = lane; v < rows >> 3; v += 32) {
        float a[8], w[8];
        load8(p.x, false, row + v * 8, a);
        load8(p.norm_w, false, k0 + v * 8, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(a[q] * w[q]));
      }
      const int ex = pow_exponent(warp_max(m));
      up = pow_up(ex);
      if (blockIdx.y == 0 && lane == 0) p.xpow[c * kLayerMaxT + warp] = pow_down(ex);
    }
    for (int v = lane; v < rows >> 3; v += 32) {
      float a[8] = {};
      if (warp < p.T) {
        float w[8];
        load8(p.x, false, row + v * 8, a);
        load8(p.norm_w, false, k0 + v * 8, w);
        __align__(16) uint16_t hi[8], lo[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          ss = fmaf(a[q], a[q], ss);
          a[q] *= w[q];
          split16<F16>(F16 ? a[q] * up : a[q], hi[q], lo[q]);
        }
        if (blockIdx.y == 0) {
          *reinterpret_cast<uint4*>(p.hi + row + v * 8) = *reinterpret_cast<uint4*>(hi);
          *reinterpret_cast<uint4*>(p.lo + row + v * 8) = *reinterpret_cast<uint4*>(lo);
        }
      }
      if (wr) {
#pragma unroll
        for (int q = 0; q < 8; ++q) xw[(v * 8 + q) * kLayerMaxT + warp] = a[q];
      }
    }
    if (blockIdx.y == 0) {
      ss = warp_sum(ss);
      if (lane == 0 && warp < p.T) p.ssq[c * kLayerMaxT + warp] = ss;
    }
  }
  if (!wr) return;
  __syncthreads();
  float acc[kLayerMaxT];
#pragma unroll
  for (int t = 0; t < kLayerMaxT; ++t) acc[t] = 0.f;
  for (int r0 = warp; r0 < rows; r0 += kRouteWarps * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + kRouteWarps * u;
      if (r < rows) {
        const float4 a = *reinterpret_cast<const float4*>(&xw[r * kLayerMaxT]);
        const float4 b = *reinterpret_cast<const float4*>(&xw[r * kLayerMaxT + 4]);
        acc[0] = fmaf(a.x, wv[u], acc[0]);
        acc[1] = fmaf(a.y, wv[u], acc[1]);
        acc[2] = fmaf(a.z, wv[u], acc[2]);
        acc[3] = fmaf(a.w, wv[u], acc[3]);
        acc[4] = fmaf(b.x, wv[u], acc[4]);
        acc[5] = fmaf(b.y, wv[u], acc[5]);
        acc[6] = fmaf(b.z, wv[u], acc[6]);
        acc[7] = fmaf(b.w, wv[u], acc[7]);
      }
      const int rn = r + kRouteWarps * U;
      wv[u] = (rn < rows && e < p.E) ? wr[(size_t)rn * p.E] : 0.f;
    }
  }
#pragma unroll
  for (int t = 0; t < kLayerMaxT; ++t) red[warp][t][lane] = acc[t];
  __syncthreads();
  if (warp < p.T && e < p.E) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) s += red[w][warp][lane];
    p.part[((size_t)c * p.T + warp) * p.E + e] = s;
  }
}

// ------------------------------------------------------------------ launch 2 --
MOE_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
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

MOE_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
MOE_DEV uint4 hmul2x4(const uint4& a, uint32_t b) {
  return make_uint4(hmul2(a.x, b), hmul2(a.y, b), hmul2(a.z, b), hmul2(a.w, b));
}

struct LayerSmem {
  int32_t ids[kLayerMaxT][kMaxTopK];
  float w[kLayerMaxT][kMaxTopK];
  float r[kLayerMaxT];
  float xpow[kLayerChunks][kLayerMaxT];
  uint8_t chunk[kLayerMaxH / 128];  // K chunk of a 128-column step
  unsigned used[kMaxExperts];       // tokens of each expert, as a bit mask
  int slot[kMaxExperts];            // its place among the active experts
  int expert[kMaxPairs];
  unsigned mask[kMaxPairs];
  int pair[kMaxPairs][kLayerMaxT];
  float wt[kMaxPairs][kLayerMaxT];
  int warp_cnt[kWarps];
  int claim[2][4];
  int flag;
  float sum[kWarps];
  int pow[kMaxPairs];  // FP8: largest exponent of the pair's intermediate
};

// Top-k of one token by one warp with the results of warp_topk (common.cuh):
// larger logit first, ties to the lower expert, NaN as -inf, softmax over the
// selected (summed in slot order), weights 0 when all of them are -inf.  Here
// the arg-max is two warp reductions of integers: the logits' bits in an
// order-preserving form, then the lowest expert that has the maximum.
template <int PER>
MOE_DEV void layer_topk(const LayerP& p, int t, int lane, float ss, LayerSmem* sm) {
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
  const float r = 1.0f / sqrtf(warp_sum(ss) / (float)p.H + p.eps);
  if (lane == 0) sm->r[t] = r;
  unsigned key[PER];  // 0: taken or beyond E
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;
    if (e < p.E) {
      float z = p.logits ? zs[i] : zs[i] * r;
      if (p.bias) z += bias[i];
      z = (z != z) ? -INFINITY : z + 0.0f;  // (-0 counts as 0)
      const unsigned u = __float_as_uint(z);
      key[i] = (u & 0x80000000u) ? ~u : u | 0x80000000u;  // -inf: 0x007fffff
    }
  }
  float sel = -INFINITY;
  int sel_e = 0;
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
    if (lane == j) {
      sel = __uint_as_float((m & 0x80000000u) ? m & 0x7fffffffu : ~m);
      sel_e = (int)at;
    }
  }
  const float top = __shfl_sync(0xffffffffu, sel, 0);
  const bool some = top > -INFINITY;
  const float e = (some && lane < p.k) ? expf(sel - top) : 0.f;
  float s = 0.f;
  for (int j = 0; j < p.k; ++j) s += __shfl_sync(0xffffffffu, e, j);
  if (lane < p.k) {
    sm->ids[t][lane] = sel_e;
    sm->w[t][lane] = some ? e / s : 0.f;
  }
}

// The tail (block_tail.cuh) of row t by the whole CTA.  `buf`: shared memory for
// the row's inputs, brought there by asynchronous copies that all run at once
// (what the tail reads was last touched before the weights went through L2), or
// nothing, when they do not fit.  The loops are kept short on purpose: this code
// runs once per launch, from a cold instruction cache.
MOE_DEV void layer_tail_row(const LayerP& p, const TailP& tail, int t, int grow, unsigned char* buf,
                            bool staged, float* red) {
  const int tid = threadIdx.x, lane = tid & 31, H = p.H, nv = H >> 3;
  const size_t row = (size_t)t * H;
  const float factor = tail_row_factor(tail, grow);
  const bool gate_row = tail.gate && tail.gate_cols != 1 && grow >= 0;
  float* f = reinterpret_cast<float*>(buf);  // [H], then h
  const unsigned char* s_res = buf + (size_t)H * 4;
  const unsigned char* s_gate = s_res + (size_t)H * 4;
  const unsigned char* s_pw = s_gate + (size_t)H * 4;
  const unsigned char* s_nw = s_pw + (size_t)H * 2;
  if (staged) cp_wait_all();
  __syncthreads();
  auto reduce = [&](float v, bool mx) {
    v = mx ? warp_max(v) : warp_sum(v);
    if (lane == 0) red[tid >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kWarps; ++w) v = mx ? fmaxf(v, red[w]) : v + red[w];
    __syncthreads();
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
    store8(tail.out, tail.out_f32 != 0, row + v * 8, h);
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
      s = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
      if (tid == 0) tail.xscale[t] = s;
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
        if (!pass && tail.xhat) store8_bf16(tail.xhat + row + v * 8, a);
      }
      if (tail.q_group) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = m > 0.f ? __fdiv_rn(m, 448.0f) : 1.0f;
        if (tail.xq && v < nv && (v & 15) == 0) tail.xscale[(size_t)t * (H >> 7) + (v >> 4)] = s;
      }
      amax = fmaxf(amax, m);
      if (tail.xq && v < nv && (pass || tail.q_group))
        *reinterpret_cast<uint2*>(tail.xq + row + v * 8) = tail_e4m3x8(a, s);
    }
  }
}

// FP8: E4M3 weights, one scale per (row >> rs) and K step * ks.
template <bool FP8, int TOK>
__global__ void __launch_bounds__(kThreadsL, 1) layer_experts_kernel(const LayerP p, const TailP tail,
                                                                     int has_tail) {
  constexpr int EB = FP8 ? 1 : 2;   // bytes per weight
  constexpr int EPC = 16 / EB;      // weights per 16-byte piece
  constexpr int KE = 64 / EB;       // K elements of a K block (64 bytes of a row)
  constexpr int Q = EPC / 8;        // 16-byte pieces of activations per K block and term
  using R = Ring<FP8, TOK>;
  constexpr int G = R::kGroups, GW = kWarps / G;  // groups, warps of a group
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ LayerSmem sm;
  __shared__ __align__(16) float red_all[kWarps * kGroupRed];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp / GW, gw = warp % GW;  // group, warp of the group
  const int g = lane >> 2, tq = lane & 3;     // MMA fragment row / column, K group
  const int T = p.T, H = p.H, E = p.E, I = p.I, k = p.k;
  sm.used[tid] = 0;
  pdl_trigger();
  __syncthreads();
  pdl_wait();

  // ---- routing (every CTA by itself; warp t: token t)
  int first_claim = 0;
  if (tid == kThreadsL - 1) first_claim = atomicAdd(&p.ctr[0], 2 * G);
  if (warp < T) {
    const float ss = lane < kLayerChunks ? __ldcg(&p.ssq[lane * kLayerMaxT + warp]) : 0.f;
    if (FP8 && lane < kLayerChunks) sm.xpow[lane][warp] = __ldcg(&p.xpow[lane * kLayerMaxT + warp]);
    if (p.ids_in) {
      if (lane < k) {
        sm.ids[warp][lane] = p.ids_in[warp * k + lane];
        sm.w[warp][lane] = p.tw_in[warp * k + lane];
      }
      const float r = 1.0f / sqrtf(warp_sum(ss) / (float)H + p.eps);
      if (lane == 0) sm.r[warp] = r;
    } else if (E <= 32) {
      layer_topk<1>(p, warp, lane, ss, &sm);
    } else if (E <= 64) {
      layer_topk<2>(p, warp, lane, ss, &sm);
    } else if (E <= 128) {
      layer_topk<4>(p, warp, lane, ss, &sm);
    } else {
      layer_topk<8>(p, warp, lane, ss, &sm);
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
  if (FP8 && warp == kWarps - 1) {
    if (lane < kLayerChunks) {
      const Chunk ch = layer_chunk(H, lane);
      for (int s = ch.k0 >> 7; s < (ch.k1 + 127) >> 7; ++s) sm.chunk[s] = (uint8_t)lane;
    }
  }
  if (tid == kThreadsL - 1) {
    for (int i = 0; i < 2 * G; ++i) sm.claim[i % G][i / G] = first_claim + i;
  }
  __syncthreads();
  // active experts in ascending order (thread e: expert e; E <= 256)
  {
    const unsigned mask = sm.used[tid];
    const unsigned act = __ballot_sync(0xffffffffu, mask != 0);
    if (lane == 0) sm.warp_cnt[warp] = __popc(act);
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
  // ones (about one per group) single, the K steps of a claim interleaved over
  // the group's warps.  FC2: output rows [n0, n1) in units of 32, all experts' K
  // steps in one sequence of which warp w takes the w-th eighth.
  const int tiles_e = I >> 3;
  const int tiles = n_act * tiles_e;
  const int singles = min(tiles, (int)(gridDim.x * G) & ~1);
  const int pairs = (tiles - singles) >> 1;  // tiles and singles are even
  const int claims = pairs + singles;
  const int n0 = (int)((int64_t)blockIdx.x * H / gridDim.x);
  const int n1 = (int)((int64_t)(blockIdx.x + 1) * H / gridDim.x);
  const uint32_t rb1 = (uint32_t)H * EB, rb2 = (uint32_t)I * EB;  // bytes of a weight row
  const int S1 = (int)((rb1 + 127) >> 7), S2 = (int)((rb2 + 127) >> 7);  // 128-byte steps of a row
  const int kb1 = (int)(rb1 >> 6), kb2 = (int)(rb2 >> 6);                // 64-byte K blocks
  const int q0 = n_act * S2 * warp / kWarps, q1 = n_act * S2 * (warp + 1) / kWarps;  // FC2 steps
  const int a_first = q0 / S2, s_first = q0 - a_first * S2;
  const unsigned magic = 0xffffffffu / (unsigned)tiles_e;
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

  unsigned char* ring = ring_all + warp * R::kWarp;
  const uint32_t ring_u = ptx::smem_u32(ring);
  const bool col = g < T;  // this lane's column is a token
  // block scales: one row of the scale matrix per 128 weight rows, one column
  // per K step; channel scales: one per row
  const int rs = p.block_scales ? 7 : 0;
  const int kg1 = p.block_scales ? H >> 7 : 1, kg2 = p.block_scales ? I >> 7 : 1;
  const int ks = p.block_scales ? 1 : 0;

  // ---- producer: the warp's steps in the order it will use them.  A segment is
  // the warp's steps of one FC1 claim, or of one expert for one FC2 unit.
  const unsigned char* p_src = nullptr;  // this lane's first row at the next step
  uint32_t p_ts = 0, p_hs = 0;           // to the second tile, to a tile's lower 8 rows (bytes)
  unsigned p_ok = 0;                     // bit 2 * tile + half: this lane's row is wanted
  const uint16_t* p_b = nullptr;         // hi term of this lane's token at the next step
  int64_t p_lo = p.lo - p.hi;            // to the lo term (elements)
  bool p_on = false;                     // the lane's token uses the expert (and may be read)
  const float* p_sc = nullptr;           // FP8: scale of row `lane` of the step's 32 rows
  const uint8_t* p_pow = nullptr;        // FP8: the token's exponents at the step (FC2)
  bool p_sok = false;
  int p_step = 0, p_end = 0, p_kb = kb1; // next step, end of its segment, K blocks of a row
  int p_inc = GW;                        // steps to the next (FC2: 1)
  int pn = -1, pu = 0, pa = a_first - 1; // claim; FC2 unit and active expert
  int n = 0;                             // claim being used; n + 1 is known too
  bool p_fc2 = false, fc1_done = false;
  int flying = 0;                        // steps issued and not yet used
  int ready = 0;                         // of these, steps known to have arrived
  uint32_t p_at = 0, c_at = 0;           // ring offsets of the next step to issue / to use

  auto start_fc2 = [&]() {
    p_fc2 = true;
    p_kb = kb2;
    p_inc = 1;
    p_ts = 16 * rb2;
    p_hs = 8 * rb2;
    p_lo = p.act_lo - p.act_hi;
  };
  // Moves to the next segment that has a step for this warp; false when there is
  // none or it is not known yet.
  auto next_segment = [&]() -> bool {
    if (!p_fc2) {
      if (pn > n || gw >= S1) return false;
      if (sm.claim[grp][(pn + 1) & 3] >= claims) start_fc2();
    }
    if (!p_fc2) {
      ++pn;
      const int c = sm.claim[grp][pn & 3];
      int a, i0;
      claim_at(c, a, i0);
      const int e = sm.expert[a];
      p_step = gw;
      p_end = S1;
      p_src = static_cast<const unsigned char*>(p.w13) + ((size_t)e * 2 * I + i0 + g) * rb1 + p_step * 128 +
              tq * 16;
      p_ts = 8 * rb1;
      p_hs = (uint32_t)I * rb1;
      p_ok = c < pairs ? 15u : 3u;
      p_on = col && ((sm.mask[a] >> g) & 1u);
      p_b = p.hi + (size_t)(p_on ? g : 0) * H + p_step * 2 * KE + tq * EPC;
      if constexpr (FP8) {
        const int row = i0 + (lane & 7) + ((lane & 8) ? I : 0) + ((lane & 16) ? 8 : 0);
        p_sok = c < pairs || lane < 16;
        p_sc = p.s13 + ((size_t)e * (2 * I >> rs) + ((p_sok ? row : 0) >> rs)) * kg1 + p_step * ks;
      }
      return true;
    }
    if (q0 == q1 || n0 + 32 * pu >= n1) return false;
    ++pa;
    if (pa * S2 >= q1) {  // the next unit of output rows
      if (n0 + 32 * (pu + 1) >= n1) {
        --pa;
        return false;
      }
      ++pu;
      pa = a_first;
    }
    const int row0 = n0 + 32 * pu, e = sm.expert[pa];
    p_step = pa == a_first ? s_first : 0;
    p_end = min(S2, q1 - pa * S2);
    p_src = static_cast<const unsigned char*>(p.w2) + ((size_t)e * H + row0 + g) * rb2 + p_step * 128 + tq * 16;
    p_ok = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) p_ok |= (row0 + g + 8 * i < n1 ? 1u : 0u) << i;
    const int pr = sm.pair[pa][g];
    p_on = pr >= 0 && fc1_done;
    p_b = p.act_hi + (size_t)(pr >= 0 ? pr : 0) * I + p_step * 2 * KE + tq * EPC;
    if constexpr (FP8) {
      p_pow = p.act_pow + (size_t)(pr >= 0 ? pr : 0) * (I >> 3) + p_step * 16 + (tq & 1) * 8;
      p_sok = row0 + lane < n1;
      p_sc = p.s2 + ((size_t)e * (H >> rs) + ((p_sok ? row0 + lane : 0) >> rs)) * kg2 + p_step * ks;
    }
    return true;
  };
  // This lane's activations of a step into the stage at ring offset `at`.
  auto copy_b = [&](uint32_t at, const uint16_t* b, int64_t lo, const uint8_t* pw, bool two) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (FP8 && kb && !two) break;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint16_t* src = b + kb * KE + q * 8;
        const uint32_t dst = ring_u + at + kStepA + lane * 16 + (kb * 2 * Q + q) * R::kPieceB;
        cp_async16(dst, src);
        cp_async16(dst + Q * R::kPieceB, src + lo);
      }
    }
    // (lane tq of a token: the 8 exponents of K block tq)
    if (FP8 && pw && tq < (two ? 2 : 1)) cp_async8(ring_u + at + R::kPowAt + tq * 64 + g * 8, pw);
  };
  // Keeps the ring full as far as the steps are known.
  auto top_up = [&]() {
    while (flying < R::kDepth) {
      if (p_step >= p_end && !next_segment()) break;
      const uint32_t dst = ring_u + p_at + lane * 16;
      const bool two = !FP8 || 2 * p_step + 1 < p_kb;
      const unsigned char *s0 = p_src, *s1 = s0 + p_hs, *s2 = s0 + p_ts, *s3 = s2 + p_hs;
      if (p_ok == 15u && two) {
        cp_async16(dst, s0);
        cp_async16(dst + 512, s0 + 64);
        cp_async16(dst + 1024, s1);
        cp_async16(dst + 1536, s1 + 64);
        cp_async16(dst + 2048, s2);
        cp_async16(dst + 2560, s2 + 64);
        cp_async16(dst + 3072, s3);
        cp_async16(dst + 3584, s3 + 64);
      } else {
        const unsigned char* src[4] = {s0, s1, s2, s3};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((p_ok >> i) & 1u) {
            cp_async16(dst + 1024 * i, src[i]);
            if (two) cp_async16(dst + 1024 * i + 512, src[i] + 64);
          }
        }
      }
      if (p_on) copy_b(p_at, p_b, p_lo, FP8 && p_fc2 ? p_pow : nullptr, two);
      if (FP8 && p_sok) cp_async4(ring_u + p_at + R::kScaleAt + lane * 4, p_sc);
      cp_commit();
      ++flying;
      p_at = p_at == (R::kDepth - 1) * R::kStage ? 0 : p_at + R::kStage;
      p_src += p_inc * 128;
      p_b += p_inc * 2 * KE;
      if constexpr (FP8) {
        p_sc += p_inc * ks;
        p_pow += p_inc * 16;
      }
      p_step += p_inc;
    }
  };

  // One step: h/l[tile] += weights of the step * the hi / lo activations.  What
  // a lane did not copy (rows that are not wanted, tokens that do not use the
  // expert) is whatever the ring held: it only reaches sums that are not used.
  struct Acc {
    float h[2][4], l[2][4];
  };
  auto clear = [](Acc& a) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) a.h[i][j] = a.l[i][j] = 0.f;
  };
  // top: FC2 with FP8, the exponent that the activations' groups are brought to
  // (0 otherwise).
  auto multiply = [&](Acc& acc, float (&sc)[4], int top, bool second_tile, bool two) {
    if (ready > 0) --ready;
    else if (flying == R::kDepth) asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
    else cp_wait_all();
    if (FP8) __syncwarp();  // scales and exponents were copied by other lanes of the warp
    const unsigned char* st = ring + c_at + lane * 16;
    const uint4* sp = reinterpret_cast<const uint4*>(st);
    // (columns beyond TOK read another token's piece; they are not used)
    const unsigned char* bp = ring + c_at + kStepA + ((g & (TOK - 1)) * 4 + tq) * 16;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (FP8 && kb && !two) break;
      uint4 h[Q], l[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        h[q] = *reinterpret_cast<const uint4*>(bp + (kb * 2 * Q + q) * R::kPieceB);
        l[q] = *reinterpret_cast<const uint4*>(bp + (kb * 2 * Q + Q + q) * R::kPieceB);
      }
      if (FP8 && top) {
        const unsigned ex = *reinterpret_cast<const uint16_t*>(ring + c_at + R::kPowAt + kb * 64 + g * 8 + tq * 2);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int d = (int)((ex >> (8 * q)) & 255u) - top;  // <= 0: an exact power of two (0 below 2^-24)
          const __half2 f2 = __float2half2_rn(__uint_as_float((uint32_t)max(127 + d, 0) << 23));
          const uint32_t f = *reinterpret_cast<const uint32_t*>(&f2);
          h[q] = hmul2x4(h[q], f);
          l[q] = hmul2x4(l[q], f);
        }
      }
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        if (tl && !second_tile) break;
        const uint4 u0 = sp[((tl * 2 + 0) * 2 + kb) * 32], u1 = sp[((tl * 2 + 1) * 2 + kb) * 32];
        if constexpr (!FP8) {
          mma_16816<false>(acc.h[tl], u0.x, u1.x, u0.y, u1.y, h[0].x, h[0].y);
          mma_16816<false>(acc.l[tl], u0.x, u1.x, u0.y, u1.y, l[0].x, l[0].y);
          mma_16816<false>(acc.h[tl], u0.z, u1.z, u0.w, u1.w, h[0].z, h[0].w);
          mma_16816<false>(acc.l[tl], u0.z, u1.z, u0.w, u1.w, l[0].z, l[0].w);
        } else {
          const uint32_t c0[4] = {u0.x, u0.y, u0.z, u0.w}, c1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_f16(c0[m], a0, a2);
            e4m3x4_f16(c1[m], a1, a3);
            const uint4 hm = h[(m >> 1) % Q], lm = l[(m >> 1) % Q];
            mma_16816<true>(acc.h[tl], a0, a1, a2, a3, (m & 1) ? hm.z : hm.x, (m & 1) ? hm.w : hm.y);
            mma_16816<true>(acc.l[tl], a0, a1, a2, a3, (m & 1) ? lm.z : lm.x, (m & 1) ? lm.w : lm.y);
          }
        }
      }
    }
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = *reinterpret_cast<const float*>(ring + c_at + R::kScaleAt + (g + 8 * i) * 4);
      __syncwarp();  // and are overwritten by them once all have read
    }
    --flying;
    c_at = c_at == (R::kDepth - 1) * R::kStage ? 0 : c_at + R::kStage;
  };
  // tot += s * acc, s per row and f per column (bit i of `mask`: token i counts).
  // A token outside the mask gets nothing (not 0 times a weight that may not be
  // finite).
  auto fold = [&](float (&tot)[2][4], Acc& acc, const float (&s)[4], const float (&f)[2], unsigned mask) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((mask >> (2 * tq + (i & 1))) & 1u) {
          const float v = acc.h[tl][i] + acc.l[tl][i];
          tot[tl][i] = FP8 ? fmaf(s[tl * 2 + (i >> 1)] * f[i & 1], v, tot[tl][i]) : tot[tl][i] + v;
        }
    clear(acc);
  };
  auto zero = [](float (&tot)[2][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) tot[i >> 2][i & 3] = 0.f;
  };
  auto store_red = [&](float* rd, const float (&tot)[2][4]) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl) {
      float* d = rd + (tl * 16 + g) * 8 + 2 * tq;
      *reinterpret_cast<float2*>(d) = make_float2(tot[tl][0], tot[tl][1]);
      *reinterpret_cast<float2*>(d + 64) = make_float2(tot[tl][2], tot[tl][3]);
    }
  };
  auto group_sync = [&]() {
    if (G == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(32 * GW) : "memory");
  };

  // Partial sums of a warp: buffer `buf` of its group, [warps of the group][2
  // tiles][16 rows][8 tokens].
  float* red = red_all + grp * GW * kGroupRed;
  int buf = 0, my_tiles = 0;
  float sc[4] = {}, tot[2][4];
  Acc acc;
  clear(acc);
  zero(tot);

  // One loop over segments, so that the stream's code exists once: FC1 claims
  // (fc2 = false), then this warp's experts of each FC2 unit.
  bool fc2 = false;
  int u = 0, a = 0, i0 = 0;
  while (true) {
    int step, end, inc, kbs, top = 0, next_claim = claims;
    unsigned mask = 0;
    bool second = true;
    float down[2] = {1.f, 1.f};
    const int c = fc2 ? 0 : sm.claim[grp][n & 3];
    if (!fc2) {
      if (c >= claims) {
        // ---- all FC1 tiles done (each CTA's writes are visible before its count).
        // Meanwhile the first W2 steps are copied.
        if (!p_fc2) start_fc2();
        top_up();
        __syncthreads();
        if (tid == 0) {
          sm.flag = 0;
          const long long t0 = clock64();
          int seen;
          do {
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(p.ctr + 1) : "memory");
          } while (seen < tiles && clock64() - t0 < ptx::kSpinLimitCycles);
          if (seen < tiles) {
            flag_status(p.status, MOE_ERR_TIMEOUT);
            sm.flag = 1;
          }
          __threadfence();
        }
        __syncthreads();
        if (sm.flag) {
          cp_wait_all();
          return;
        }
        if constexpr (FP8) {
          if (tid < T * k) sm.pow[tid] = max(15, __ldcg(&p.ctr[kCtrPow + tid]));
        }
        // the activations of the W2 steps already in flight
        fc1_done = true;
        if (p_step < p_end) p_on = sm.pair[pa][g] >= 0;
        int qa = a_first, qs = s_first, qq = q0;
        uint32_t at = c_at;
        for (int left = flying; left > 0; --left) {
          const int pr = sm.pair[qa][g];
          if (pr >= 0)
            copy_b(at, p.act_hi + (size_t)pr * I + qs * 2 * KE + tq * EPC, p.act_lo - p.act_hi,
                   FP8 ? p.act_pow + (size_t)pr * (I >> 3) + qs * 16 + (tq & 1) * 8 : nullptr,
                   2 * qs + 1 < kb2);
          at = at == (R::kDepth - 1) * R::kStage ? 0 : at + R::kStage;
          if (++qq == q1) {  // (a short unit: the next one's steps follow)
            qa = a_first;
            qs = s_first;
            qq = q0;
          } else if (++qs == S2) {
            ++qa;
            qs = 0;
          }
        }
        cp_wait_all();
        ready = flying;
        __syncthreads();
        fc2 = true;
        buf = 0;
        a = a_first;
        continue;
      }
      claim_at(c, a, i0);
      mask = sm.mask[a];
      second = c < pairs;
      step = gw;
      end = S1;
      inc = GW;
      kbs = kb1;
      if (gw == 0 && lane == 0) next_claim = atomicAdd(&p.ctr[0], 1);  // used two claims from here
    } else {
      if (n0 + 32 * u >= n1) break;
      second = n0 + 32 * u + 16 < n1;
      inc = 1;
      kbs = kb2;
      step = a == a_first ? s_first : 0;
      end = min(S2, q1 - a * S2);  // (nothing for a warp without steps)
      if (step < end) {
        mask = sm.mask[a];
        if constexpr (FP8) {  // the pair's exponent of the lane's token, and its power for the two columns
          const int pr = sm.pair[a][g], c0 = sm.pair[a][2 * tq], c1 = sm.pair[a][2 * tq + 1];
          top = pr >= 0 ? sm.pow[pr] : 15;
          if (c0 >= 0) down[0] = pow_down(sm.pow[c0]);
          if (c1 >= 0) down[1] = pow_down(sm.pow[c1]);
        }
      }
    }
#pragma unroll 1
    for (; step < end; step += inc) {
      top_up();
      multiply(acc, sc, top, second, 2 * step + 1 < kbs);
      if constexpr (FP8) {
        if (!fc2) {
          const float2 d = *reinterpret_cast<const float2*>(&sm.xpow[sm.chunk[step]][2 * tq]);
          down[0] = d.x;
          down[1] = d.y;
        }
        fold(tot, acc, sc, down, mask);
      }
    }
    if constexpr (!FP8) fold(tot, acc, sc, down, mask);
    if (fc2 && (a + 1) * S2 < q1) {  // the unit's next expert
      ++a;
      continue;
    }
    float* rd = red + buf * (GW * kGroupRed / 2);
    if (fc2) {
      // ---- the unit's output rows: the partial sums of all warps
      rd = red_all + buf * (kWarps * kGroupRed / 2);
      store_red(rd + warp * 256, tot);
      zero(tot);
      __syncthreads();
      const int row = n0 + 32 * u + lane, t = warp;
      if (t < T && row < n1) {
        const float* s = rd + lane * 8 + t;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += s[w * 256];
        const size_t at = (size_t)t * H + row;
        if (has_tail) p.f[at] = v;
        else static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(v);
      }
      ++u;
      a = a_first;
    } else {
      // ---- the claim's intermediate columns: 16 lanes a token
      store_red(rd + gw * 256, tot);
      zero(tot);
      if (gw == 0 && lane == 0) sm.claim[grp][(n + 2) & 3] = next_claim;
      group_sync();
      const int il = lane & 15;
      // G = 1: warp t, token t, each half warp half of the partial sums;
      // G = 2: two tokens a warp
      const int t = G == 1 ? gw : 2 * gw + (lane >> 4);
      if (G == 1 ? (mask >> t) & 1u : (mask >> (2 * gw)) & 3u) {
        const float* s = rd + ((il >> 3) * 16 + (il & 7)) * 8 + t + (G == 1 ? (lane >> 4) * 1024 : 0);
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          gate += s[w * 256];
          up += s[w * 256 + 64];
        }
        if (G == 1) {
          gate += __shfl_xor_sync(0xffffffffu, gate, 16);
          up += __shfl_xor_sync(0xffffffffu, up, 16);
        }
        const bool mine = ((mask >> t) & 1u) && il < (second ? 16 : 8) && (G == 2 || lane < 16);
        const float r = sm.r[t];
        // the routing weight goes into the intermediate, so FC2 adds the token's
        // experts without a factor
        float v = silu_f(gate * r) * (up * r) * sm.wt[a][t];
        const int pr = max(sm.pair[a][t], 0);
        if constexpr (FP8) {  // eight columns share a power of two
          float m = fabsf(v);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int ex = pow_exponent(m);
          if (mine && (il & 7) == 0) {
            p.act_pow[(size_t)pr * (I >> 3) + (i0 + il) / 8] = (uint8_t)ex;
            atomicMax(&p.ctr[kCtrPow + pr], ex);
          }
          v *= pow_up(ex);
        }
        if (mine) {
          const size_t at = (size_t)pr * I + i0 + il;
          split16<FP8>(v, p.act_hi[at], p.act_lo[at]);
        }
      }
      my_tiles += second ? 2 : 1;
      // the group's last claim: its tiles are counted once its writes are there
      if (sm.claim[grp][(n + 1) & 3] >= claims) {
        group_sync();
        if (gw == 0 && lane == 0) {
          __threadfence();
          atomicAdd(&p.ctr[1], my_tiles);
        }
      }
      ++n;
    }
    buf ^= 1;
  }
  cp_wait_all();
  if (!has_tail) return;

  // ---- tail: the last T CTAs to finish take a row each.  (When they wait for
  // one another, fewer than T CTAs are unfinished, and the others have left their
  // SMs to them.)
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    sm.flag = atomicAdd(&p.ctr[2], 1) - ((int)gridDim.x - T);
  }
  __syncthreads();
  const int t = sm.flag;
  if (t < 0) return;
  const int grow = tail_gate_row(tail, t, tid == 0 ? p.status : nullptr);
  // the row's inputs into the ring's shared memory: f [H] fp32, residual, gate
  // row (room for fp32 each), the norms' weights
  const bool staged = (size_t)H * 16 <= (size_t)R::kBytes;
  static_assert(kLayerMaxH * 4 <= R::kBytes, "f fits in any case");
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
  __syncthreads();
  stage(0, p.f + (size_t)t * H, (size_t)H * 4);
  cp_wait_all();
  layer_tail_row(p, tail, t, grow, ring_all, staged, sm.sum);
}

struct LayerWs {
  size_t hi, lo, ssq, xpow, part, ctr, act_hi, act_lo, act_pow, f, total;
};

LayerWs layer_layout(int T, int H, int E, int I, int k) {
  LayerWs w{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~(size_t)255;
    return at;
  };
  const size_t t = T > 0 ? T : 1;
  w.hi = take(t * H * 2);
  w.lo = take(t * H * 2);
  w.ssq = take((size_t)kLayerChunks * kLayerMaxT * 4);
  w.xpow = take((size_t)kLayerChunks * kLayerMaxT * 4);
  w.part = take((size_t)kLayerChunks * t * E * 4);
  w.ctr = take(kCtrInts * 4);
  w.act_hi = take(t * k * I * 2);
  w.act_lo = take(t * k * I * 2);
  w.act_pow = take(t * k * (I / 8));
  w.f = take(t * H * 4);
  w.total = o;
  return w;
}

}  // namespace

size_t layer_workspace_bytes(int T, int H, int E, int I, int k) {
  return layer_layout(T, H, E, I, k).total;
}

cudaError_t launch_layer(const LayerArgs& a, const TailP* tail, int sms, int* status, cudaStream_t st) {
  const LayerWs w = layer_layout(a.T, a.H, a.E, a.I, a.k);
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
  p.hi = reinterpret_cast<uint16_t*>(ws + w.hi);
  p.lo = reinterpret_cast<uint16_t*>(ws + w.lo);
  p.act_hi = reinterpret_cast<uint16_t*>(ws + w.act_hi);
  p.act_lo = reinterpret_cast<uint16_t*>(ws + w.act_lo);
  p.act_pow = ws + w.act_pow;
  p.ssq = reinterpret_cast<float*>(ws + w.ssq);
  p.xpow = reinterpret_cast<float*>(ws + w.xpow);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.f = reinterpret_cast<float*>(ws + w.f);
  p.ctr = reinterpret_cast<int*>(ws + w.ctr);
  p.status = status;
  int rows = 0;  // of the largest chunk
  for (int c = 0; c < kLayerChunks; ++c) {
    const Chunk ch = layer_chunk(a.H, c);
    if (ch.k1 - ch.k0 > rows) rows = ch.k1 - ch.k0;
  }
  const int route_smem = a.router_w ? rows * kLayerMaxT * 4 : 0;  // up to 32 KB beside the static part
  auto route = a.fp8 ? layer_route_kernel<true> : layer_route_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (route_smem > (24 << 10))
    e = cudaFuncSetAttribute(route, cudaFuncAttributeMaxDynamicSharedMemorySize, route_smem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(route, dim3(kLayerChunks, a.router_w ? (a.E + 31) / 32 : 1), dim3(32 * kRouteWarps),
                    (size_t)route_smem, st, p);
  if (e != cudaSuccess) return e;
  auto kern = a.fp8 ? layer_experts_kernel<true, 8> : layer_experts_kernel<false, 8>;
  int smem = a.fp8 ? Ring<true, 8>::kBytes : Ring<false, 8>::kBytes;
  if (a.T <= 4) {
    kern = a.fp8 ? layer_experts_kernel<true, 4> : layer_experts_kernel<false, 4>;
    smem = a.fp8 ? Ring<true, 4>::kBytes : Ring<false, 4>::kBytes;
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(sms), dim3(kThreadsL), smem, st, p, tail ? *tail : TailP{},
                       tail ? 1 : 0);
}

}  // namespace moe
