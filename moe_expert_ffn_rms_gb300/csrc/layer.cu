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
// Launch 1 (layer_route_kernel) multiplies x by the norm weight, splits it for
// the products, and takes the router's partial dot products and the partial
// sums of squares per K chunk.  r is a factor of the row, so it is applied
// afterwards, to the logits and to the FC1 results, and nothing in this launch
// waits for a whole row.
//
// Launch 2 (layer_experts_kernel), one persistent CTA per SM: every CTA adds the
// partial logits and picks the experts by itself, takes FC1 row tiles of the
// active experts from a counter, waits until all tiles are done, and computes
// its own slice of H output rows over all experts -- the sum over a token's
// experts stays in its accumulators.  The CTA that finishes last does the tail.
// Claiming the FC1 tiles from a counter means the wait needs no co-residency:
// a CTA that has not started holds no tile.
//
// Products: the weights are the 16 x 16 operand of m16n8k16 bf16 MMAs, the (at
// most 8) tokens the 8 columns.  Activations enter as two bf16 terms hi + lo
// (16 bits of mantissa), so neither x_hat nor the intermediate is rounded to
// bf16; accumulation is fp32.  A warp reads its own operands: each lane copies
// exactly the 16-byte pieces it will feed to its MMAs into its own part of
// shared memory (cp.async, a few steps ahead) and reads them back, so the
// stream needs no barrier, and the first W2 pieces are already on their way
// while the CTA waits for the other CTAs' FC1 tiles.  The order of the K
// elements inside a piece is the same for both operands and therefore free.
// The activations go the same way as the weights: a plain load of them would
// wait behind the copies in flight (4 us of them with 160 KB per SM).
//
// mma.sync and not tcgen05: at 8 columns the tensor work is 1/16 of what the
// legacy instruction sustains at this memory rate, a fragment load straight from
// the copied bytes needs no descriptor layout, and accumulators in registers
// spare the TMEM round trip between short row tiles.
#include "block_tail.cuh"
#include "kernels.h"
#include "tail.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsL = 32 * kWarps;

// Per-warp stage of the copy ring: weights [2 tiles][2 row halves][2 K blocks]
// [32 lanes] of 16 bytes; activations [2 K blocks][hi, lo][pieces][8 tokens]
// [4 lanes] of 16 bytes; FP8: the scales of the 32 rows.  Three steps of eight
// warps keep 96 KB per SM in flight, which already streams at the copy
// bandwidth (measured alone: 6.64 TB/s with 3 steps, 6.64 with 6).
constexpr int kStepA = 4096;
constexpr int kPieceB = 512;
template <bool FP8>
struct Ring {
  static constexpr int kScaleAt = kStepA + 4 * (FP8 ? 2 : 1) * kPieceB;
  static constexpr int kStage = kScaleAt + (FP8 ? 128 : 0);
  static constexpr int kDepth = FP8 ? 3 : 4;
  static constexpr int kWarp = kDepth * kStage;
  static constexpr int kBytes = kWarps * kWarp;  // 192 KB, 195 KB
};
constexpr int kRedFloats = kWarps * 2 * 16 * 8; // partial sums of two row tiles
constexpr int kMaxPairs = kLayerMaxT * kMaxTopK;

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
  bf16 *hi, *lo, *act_hi, *act_lo;
  float *ssq, *part, *f;
  int* ctr;  // [0] FC1 claims, [1] FC1 tiles done, [2] CTAs finished
  int* status;
};

// ------------------------------------------------------------------ launch 1 --
// Grid (kLayerChunks, groups of 32 experts): K chunk c, experts 32y .. 32y+31.
// Latency is all there is: each warp has its rows of W_r (16 at H = 4096) on
// their way before it waits for anything.
constexpr int kRouteWarps = 16;

__global__ void __launch_bounds__(32 * kRouteWarps) layer_route_kernel(const LayerP p) {
  extern __shared__ __align__(16) float xw[];  // [rows of the chunk][8 tokens]
  __shared__ float red[kRouteWarps][kLayerMaxT][32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x, nb = p.H >> 3;
  const int b0 = (int)((int64_t)c * nb / kLayerChunks), b1 = (int)((int64_t)(c + 1) * nb / kLayerChunks);
  const int k0 = b0 * 8, rows = (b1 - b0) * 8;
  if (c == 0 && blockIdx.y == 0 && tid < 4) p.ctr[tid] = 0;
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
    float ss = 0.f;
    for (int v = lane; v < b1 - b0; v += 32) {
      float a[8] = {}, hi[8], lo[8];
      if (warp < p.T) {
        float w[8];
        load8(p.x, false, (size_t)warp * p.H + k0 + v * 8, a);
        load8(p.norm_w, false, k0 + v * 8, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          ss = fmaf(a[q], a[q], ss);
          a[q] *= w[q];
          hi[q] = bf16_round_f(a[q]);
          lo[q] = a[q] - hi[q];
        }
        if (blockIdx.y == 0) {
          store8_bf16(p.hi + (size_t)warp * p.H + k0 + v * 8, hi);
          store8_bf16(p.lo + (size_t)warp * p.H + k0 + v * 8, lo);
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
MOE_DEV void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
MOE_DEV void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes as two bf16 pairs (every E4M3 value is exact in bf16).
MOE_DEV void e4m3x4_bf16(uint32_t q, uint32_t& lo, uint32_t& hi) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q & 0xffffu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> 16), __NV_E4M3);
  const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
  lo = pack2_bf16(fa.x, fa.y);
  hi = pack2_bf16(fb.x, fb.y);
}

struct LayerSmem {
  int32_t ids[kLayerMaxT][kMaxTopK];
  float w[kLayerMaxT][kMaxTopK];
  float r[kLayerMaxT];
  unsigned used[kMaxExperts];  // tokens of each expert, as a bit mask
  int slot[kMaxExperts];       // its place among the active experts
  int expert[kMaxPairs];
  unsigned mask[kMaxPairs];
  int pair[kMaxPairs][kLayerMaxT];
  float wt[kMaxPairs][kLayerMaxT];
  int warp_cnt[kWarps];
  int claim[4];
  int flag;
  float sum[kWarps];
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

// FP8: E4M3 weights, one scale per (row >> rs) and K step * ks.
template <bool FP8>
__global__ void __launch_bounds__(kThreadsL, 1) layer_experts_kernel(const LayerP p, const TailP tail,
                                                                     int has_tail) {
  constexpr int EB = FP8 ? 1 : 2;   // bytes per weight
  constexpr int EPC = 16 / EB;      // weights per 16-byte piece
  constexpr int KE = 64 / EB;       // K elements of a K block (64 bytes of a row)
  constexpr int Q = EPC / 8;        // 16-byte pieces of activations per K block and term
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ LayerSmem sm;
  __shared__ __align__(16) float red[2][kRedFloats];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tq = lane & 3;  // MMA fragment row / column, K group
  const int T = p.T, H = p.H, E = p.E, I = p.I, k = p.k;
  sm.used[tid] = 0;
  pdl_trigger();
  __syncthreads();
  pdl_wait();

  // ---- routing (every CTA by itself; warp t: token t)
  int first_claim = 0;
  if (tid == kThreadsL - 1) first_claim = atomicAdd(&p.ctr[0], 2);
  if (has_tail) {  // what the tail will read is brought to L2 meanwhile
    const int64_t line = (int64_t)blockIdx.x * kThreadsL + tid;
    auto warm = [&](const void* q, int64_t bytes) {
      if (q && line * 128 < bytes)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(q) + line * 128));
    };
    warm(tail.residual, (int64_t)T * H * (tail.res_f32 ? 4 : 2));
    warm(tail.post_w, 2 * H);
    warm(tail.next_w, 2 * H);
    if (tail.gate_cols == H && tail.gate_rows == 1) warm(tail.gate, (int64_t)H * (tail.gate_f32 ? 4 : 2));
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
  if (tid == kThreadsL - 1) {
    sm.claim[0] = first_claim;
    sm.claim[1] = first_claim + 1;
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

  // ---- work: FC1 row tiles (8 gate + 8 up rows) in claims of two, the last
  // ones (one per CTA) single; FC2 output rows [n0, n1) in units of 32
  const int tiles_e = I >> 3;
  const int tiles = n_act * tiles_e;
  const int singles = min(tiles, (int)gridDim.x & ~1);
  const int pairs = (tiles - singles) >> 1;  // tiles and singles are even
  const int claims = pairs + singles;
  const int n0 = (int)((int64_t)blockIdx.x * H / gridDim.x);
  const int n1 = (int)((int64_t)(blockIdx.x + 1) * H / gridDim.x);
  const uint32_t rb1 = (uint32_t)H * EB, rb2 = (uint32_t)I * EB;  // bytes of a weight row
  const int S1 = (int)((rb1 + 127) >> 7), S2 = (int)((rb2 + 127) >> 7);  // 128-byte steps of a row
  const int kb1 = (int)(rb1 >> 6), kb2 = (int)(rb2 >> 6);                // 64-byte K blocks
  auto claim_tile = [&](int c) { return c < pairs ? 2 * c : c + pairs; };

  using R = Ring<FP8>;
  unsigned char* ring = ring_all + warp * R::kWarp;
  const uint32_t ring_u = ptx::smem_u32(ring);
  const bool col = g < T;  // this lane's column is a token
  // block scales: one row of the scale matrix per 128 weight rows, one column
  // per K step; channel scales: one per row
  const int rs = p.block_scales ? 7 : 0;
  const int kg1 = p.block_scales ? H >> 7 : 1, kg2 = p.block_scales ? I >> 7 : 1;
  const int ks = p.block_scales ? 1 : 0;

  // ---- producer: the warp's steps in the order it will use them.  A segment is
  // the warp's steps of one FC1 claim, or of one expert for one FC2 unit; step
  // q of all experts' steps goes to warp q mod 8.
  const unsigned char* p_src = nullptr;  // this lane's first row at the next step
  uint32_t p_ts = 0, p_hs = 0;           // to the second tile, to a tile's lower 8 rows (bytes)
  unsigned p_ok = 0;                     // bit 2 * tile + half: this lane's row is wanted
  const bf16* p_b = nullptr;             // hi term of this lane's token at the next step
  int64_t p_lo = 0;                      // to the lo term (elements)
  bool p_on = false;                     // the lane's token uses the expert (and may be read)
  const float* p_sc = nullptr;           // FP8: scale of row `lane` of the step's 32 rows
  bool p_sok = false;
  int p_step = 0, p_end = 0, p_kb = 0;   // next step, steps and K blocks of a row
  int pn = -1, pu = 0, pa = -1;          // claim; FC2 unit and active expert
  int known = 1;                         // newest claim index published to this warp
  bool p_fc2 = false, fc1_done = false;
  int flying = 0;                        // steps issued and not yet used
  int ready = 0;                         // of these, steps known to have arrived
  uint32_t p_at = 0, c_at = 0;           // ring offsets of the next step to issue / to use

  // Moves to the next segment that has a step for this warp.
  auto next_segment = [&]() -> bool {
    while (!p_fc2) {
      if (pn + 1 > known) return false;
      const int c = sm.claim[(pn + 1) & 3];
      if (c >= claims) {
        p_fc2 = true;
        break;
      }
      ++pn;
      if (warp >= S1) continue;
      const int tile = claim_tile(c), a = tile / tiles_e;
      const int i0 = (tile - a * tiles_e) * 8;
      const int e = sm.expert[a];
      p_step = warp;
      p_end = S1;
      p_kb = kb1;
      p_src = static_cast<const unsigned char*>(p.w13) + ((size_t)e * 2 * I + i0 + g) * rb1 + p_step * 128 +
              tq * 16;
      p_ts = 8 * rb1;
      p_hs = (uint32_t)I * rb1;
      p_ok = c < pairs ? 15u : 3u;
      p_on = col && ((sm.mask[a] >> g) & 1u);
      p_b = p.hi + (size_t)(p_on ? g : 0) * H + p_step * 2 * KE + tq * EPC;
      p_lo = p.lo - p.hi;
      if constexpr (FP8) {
        const int row = i0 + (lane & 7) + ((lane & 8) ? I : 0) + ((lane & 16) ? 8 : 0);
        p_sok = c < pairs || lane < 16;
        p_sc = p.s13 + ((size_t)e * (2 * I >> rs) + ((p_sok ? row : 0) >> rs)) * kg1 + p_step * ks;
      }
      return true;
    }
    while (n0 + 32 * pu < n1) {
      if (++pa >= n_act) {
        if (n_act == 0) return false;
        pa = -1;
        ++pu;
        continue;
      }
      p_step = (warp - pa * S2) & (kWarps - 1);
      if (p_step >= S2) continue;
      const int row0 = n0 + 32 * pu, e = sm.expert[pa];
      p_end = S2;
      p_kb = kb2;
      p_src = static_cast<const unsigned char*>(p.w2) + ((size_t)e * H + row0 + g) * rb2 + p_step * 128 +
              tq * 16;
      p_ts = 16 * rb2;
      p_hs = 8 * rb2;
      p_ok = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) p_ok |= (row0 + g + 8 * i < n1 ? 1u : 0u) << i;
      const int pr = sm.pair[pa][g];
      p_on = pr >= 0 && fc1_done;
      p_b = p.act_hi + (size_t)(pr >= 0 ? pr : 0) * I + p_step * 2 * KE + tq * EPC;
      p_lo = p.act_lo - p.act_hi;
      if constexpr (FP8) {
        p_sok = row0 + lane < n1;
        p_sc = p.s2 + ((size_t)e * (H >> rs) + ((p_sok ? row0 + lane : 0) >> rs)) * kg2 + p_step * ks;
      }
      return true;
    }
    p_end = 0;
    return false;
  };
  // This lane's activations of a step into the stage at ring offset `at`.
  auto copy_b = [&](uint32_t at, const bf16* b, int64_t lo, bool two) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (FP8 && kb && !two) break;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const bf16* src = b + kb * KE + q * 8;
        const uint32_t dst = ring_u + at + kStepA + lane * 16 + (kb * 2 * Q + q) * kPieceB;
        cp_async16(dst, src);
        cp_async16(dst + Q * kPieceB, src + lo);
      }
    }
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
      if (p_on) copy_b(p_at, p_b, p_lo, two);
      if (FP8 && p_sok) cp_async4(ring_u + p_at + R::kScaleAt + lane * 4, p_sc);
      cp_commit();
      ++flying;
      p_at = p_at == (R::kDepth - 1) * R::kStage ? 0 : p_at + R::kStage;
      p_src += kWarps * 128;
      p_b += kWarps * 2 * KE;
      p_sc += kWarps * ks;
      p_step += kWarps;
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
  auto multiply = [&](Acc& acc, float (&sc)[4], bool second_tile, bool two) {
    if (ready > 0) --ready;
    else if (flying == R::kDepth) asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
    else asm volatile("cp.async.wait_all;" ::: "memory");
    const unsigned char* st = ring + c_at + lane * 16;
    const uint4* sp = reinterpret_cast<const uint4*>(st);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (FP8 && kb && !two) break;
      uint4 h[Q], l[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        h[q] = *reinterpret_cast<const uint4*>(st + kStepA + (kb * 2 * Q + q) * kPieceB);
        l[q] = *reinterpret_cast<const uint4*>(st + kStepA + (kb * 2 * Q + Q + q) * kPieceB);
      }
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        if (tl && !second_tile) break;
        const uint4 u0 = sp[((tl * 2 + 0) * 2 + kb) * 32], u1 = sp[((tl * 2 + 1) * 2 + kb) * 32];
        if constexpr (!FP8) {
          mma_16816(acc.h[tl], u0.x, u1.x, u0.y, u1.y, h[0].x, h[0].y);
          mma_16816(acc.l[tl], u0.x, u1.x, u0.y, u1.y, l[0].x, l[0].y);
          mma_16816(acc.h[tl], u0.z, u1.z, u0.w, u1.w, h[0].z, h[0].w);
          mma_16816(acc.l[tl], u0.z, u1.z, u0.w, u1.w, l[0].z, l[0].w);
        } else {
          const uint32_t q0[4] = {u0.x, u0.y, u0.z, u0.w}, q1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_bf16(q0[m], a0, a2);
            e4m3x4_bf16(q1[m], a1, a3);
            const uint4 hm = h[(m >> 1) % Q], lm = l[(m >> 1) % Q];
            mma_16816(acc.h[tl], a0, a1, a2, a3, (m & 1) ? hm.z : hm.x, (m & 1) ? hm.w : hm.y);
            mma_16816(acc.l[tl], a0, a1, a2, a3, (m & 1) ? lm.z : lm.x, (m & 1) ? lm.w : lm.y);
          }
        }
      }
    }
    if constexpr (FP8) {
      __syncwarp();  // the scales were copied by other lanes of the warp
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[i] = *reinterpret_cast<const float*>(ring + c_at + R::kScaleAt + (g + 8 * i) * 4);
      __syncwarp();  // and are overwritten by them once all have read
    }
    --flying;
    c_at = c_at == (R::kDepth - 1) * R::kStage ? 0 : c_at + R::kStage;
  };
  auto store_red = [&](float* rd, const float (&tot)[2][4]) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl) {
      float* d = rd + ((warp * 2 + tl) * 16 + g) * 8 + 2 * tq;
      *reinterpret_cast<float2*>(d) = make_float2(tot[tl][0], tot[tl][1]);
      *reinterpret_cast<float2*>(d + 64) = make_float2(tot[tl][2], tot[tl][3]);
    }
  };
  // tot += s * acc, s per row (bit i of `mask`: token i counts).  A token outside
  // the mask gets nothing (not 0 times a weight that may not be finite).
  auto fold = [&](float (&tot)[2][4], const Acc& acc, const float (&s)[4], unsigned mask) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((mask >> (2 * tq + (i & 1))) & 1u) {
          const float v = acc.h[tl][i] + acc.l[tl][i];
          tot[tl][i] = FP8 ? fmaf(s[tl * 2 + (i >> 1)], v, tot[tl][i]) : tot[tl][i] + v;
        }
  };

  int buf = 0;
  int my_tiles = 0;
  float sc[4] = {};

  // ---- FC1
  for (int n = 0;; ++n) {
    const int c = sm.claim[n & 3];
    if (c >= claims) break;
    int next_claim = claims;
    if (tid == 0) next_claim = atomicAdd(&p.ctr[0], 1);  // used two claims from here
    const int tile = claim_tile(c), a = tile / tiles_e;
    const bool two_tiles = c < pairs;
    const int i0 = (tile - a * tiles_e) * 8;
    const unsigned mask = sm.mask[a];
    float tot[2][4] = {};
    Acc acc;
    clear(acc);
    for (int step = warp; step < S1; step += kWarps) {
      top_up();
      multiply(acc, sc, two_tiles, 2 * step + 1 < kb1);
      if constexpr (FP8) {
        fold(tot, acc, sc, mask);
        clear(acc);
      }
    }
    if constexpr (!FP8) fold(tot, acc, sc, mask);
    store_red(red[buf], tot);
    if (tid == 0) sm.claim[(n + 2) & 3] = next_claim;
    __syncthreads();
    known = n + 2;
    // warp t: the 16 intermediate columns of token t (each half warp adds four
    // warps' partial sums)
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
      if (lane < (two_tiles ? 16 : 8)) {
        const float r = sm.r[warp];
        // the routing weight goes into the intermediate, so FC2 adds the
        // token's experts without a factor
        const float v = silu_f(gate * r) * (up * r) * sm.wt[a][warp];
        const float hi = bf16_round_f(v);
        const size_t at = (size_t)sm.pair[a][warp] * I + i0 + il;
        p.act_hi[at] = __float2bfloat16_rn(hi);
        p.act_lo[at] = __float2bfloat16_rn(v - hi);
      }
    }
    my_tiles += two_tiles ? 2 : 1;
    buf ^= 1;
  }
  // ---- all FC1 tiles done (each CTA's writes are visible before its count);
  // the first W2 steps are copied meanwhile
  top_up();
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (my_tiles) atomicAdd(&p.ctr[1], my_tiles);
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
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  // the activations of the steps already in flight (the warp's first ones)
  fc1_done = true;
  if (p_step < p_end) p_on = sm.pair[pa][g] >= 0;
  {
    int a = -1, step = S2;
    uint32_t at = c_at;
    for (int left = flying; left > 0; --left) {
      step += kWarps;
      while (step >= S2) {
        if (++a == n_act) a = 0;  // (a short unit: the next one's steps follow)
        step = (warp - a * S2) & (kWarps - 1);
      }
      const int pr = sm.pair[a][g];
      if (pr >= 0)
        copy_b(at, p.act_hi + (size_t)pr * I + step * 2 * KE + tq * EPC, p.act_lo - p.act_hi,
               2 * step + 1 < kb2);
      at = at == (R::kDepth - 1) * R::kStage ? 0 : at + R::kStage;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    ready = flying;
  }

  // ---- FC2: this CTA's output rows over all active experts
  for (int u = 0; n0 + 32 * u < n1; ++u) {
    const int row0 = n0 + 32 * u;
    const bool second = row0 + 16 < n1;
    float tot[2][4] = {};
    Acc acc;
    clear(acc);
    for (int a = 0; a < n_act; ++a) {
      const unsigned mask = sm.mask[a];
      for (int step = (warp - a * S2) & (kWarps - 1); step < S2; step += kWarps) {
        top_up();
        multiply(acc, sc, second, 2 * step + 1 < kb2);
        if constexpr (FP8) {
          fold(tot, acc, sc, mask);
          clear(acc);
        }
      }
      if constexpr (!FP8) {
        fold(tot, acc, sc, mask);
        clear(acc);
      }
    }
    store_red(red[buf], tot);
    __syncthreads();
    const int row = lane, t = warp;
    if (t < T && row0 + row < n1) {
      const float* s = red[buf] + row * 8 + t;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s[w * 256];
      const size_t at = (size_t)t * H + row0 + row;
      if (has_tail) p.f[at] = v;
      else static_cast<bf16*>(p.out)[at] = __float2bfloat16_rn(v);
    }
    buf ^= 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!has_tail) return;

  // ---- tail: the CTA that finishes last takes all rows; 256 / Tp threads per
  // row (Tp: T rounded up to a power of two), eight columns a thread at a time.
  const int tp = T <= 1 ? 1 : (T <= 2 ? 2 : (T <= 4 ? 4 : 8));
  const int ntr = kThreadsL / tp, wpr = kWarps / tp;
  const int t = tid / ntr, sub = tid - t * ntr;
  const bool on = t < T;
  const int nv = H >> 3;
  // What a thread's first kPre pieces need besides f is loaded before the CTA
  // knows whether it is the last.
  constexpr int kPre = 2;
  float pre_res[kPre][8] = {};
  uint4 pre_pw[kPre] = {}, pre_nw[kPre] = {};
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    const int v = sub + i * ntr;
    if (on && v < nv) {
      if (tail.residual) load8(tail.residual, tail.res_f32 != 0, (size_t)t * H + v * 8, pre_res[i]);
      if (tail.post_w) pre_pw[i] = reinterpret_cast<const uint4*>(tail.post_w)[v];
      if (tail.next_w) pre_nw[i] = reinterpret_cast<const uint4*>(tail.next_w)[v];
    }
  }
  const int grow = on ? tail_gate_row(tail, t, nullptr) : 0;
  const float factor = on ? tail_row_factor(tail, grow) : 0.f;
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    sm.flag = atomicAdd(&p.ctr[2], 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!sm.flag) return;
  if (grow < 0 && sub == 0) flag_status(p.status, MOE_ERR_INVALID_ARG);
  // The rows are kept in the ring's shared memory between the passes where they
  // fit (a thread reads back only what it wrote).
  float* keep = (size_t)T * H * 4 <= (size_t)R::kBytes ? reinterpret_cast<float*>(ring_all) : p.f;
  auto kept = [&](int v) { return reinterpret_cast<float4*>(keep + (size_t)t * H + v * 8); };
  auto row_reduce = [&](float v, bool mx) {
    v = mx ? warp_max(v) : warp_sum(v);
    if (lane == 0) sm.sum[warp] = v;
    __syncthreads();
    v = sm.sum[t * wpr];
    for (int w = 1; w < wpr; ++w) v = mx ? fmaxf(v, sm.sum[t * wpr + w]) : v + sm.sum[t * wpr + w];
    __syncthreads();
    return v;
  };
  float ss = 0.f;
  if (on) {
#pragma unroll 4
    for (int v = sub; v < nv; v += ntr) {
      const float4* s = reinterpret_cast<const float4*>(p.f + (size_t)t * H + v * 8);
      const float4 a = __ldcg(s), b = __ldcg(s + 1);
      kept(v)[0] = a;
      kept(v)[1] = b;
      ss += a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w;
    }
  }
  const float r = tail.post_w ? 1.0f / sqrtf(row_reduce(ss, false) / (float)H + tail.post_eps) : 1.f;
  ss = 0.f;
  auto residual8 = [&](int v, const float (&res)[8], const uint4& pw) {
    float f[8], w[8], h[8];
    load8(kept(v), true, 0, f);
    unpack8_bf16(pw, w);
    tail_h8(tail, H, v * 8, f, w, r, grow, factor, res, h);
    store8(tail.out, tail.out_f32 != 0, (size_t)t * H + v * 8, h);
    kept(v)[0] = make_float4(h[0], h[1], h[2], h[3]);
    kept(v)[1] = make_float4(h[4], h[5], h[6], h[7]);
#pragma unroll
    for (int q = 0; q < 8; ++q) ss = fmaf(h[q], h[q], ss);
  };
  if (on) {
#pragma unroll
    for (int i = 0; i < kPre; ++i)
      if (sub + i * ntr < nv) residual8(sub + i * ntr, pre_res[i], pre_pw[i]);
#pragma unroll 2
    for (int v = sub + kPre * ntr; v < nv; v += ntr) {
      float res[8] = {};
      uint4 pw = make_uint4(0u, 0u, 0u, 0u);
      if (tail.residual) load8(tail.residual, tail.res_f32 != 0, (size_t)t * H + v * 8, res);
      if (tail.post_w) pw = reinterpret_cast<const uint4*>(tail.post_w)[v];
      residual8(v, res, pw);
    }
  }
  if (!tail.next_w) return;
  const float rn = 1.0f / sqrtf(row_reduce(ss, false) / (float)H + tail.next_eps);
  float amax = 0.f;
  auto next8 = [&](int v, const uint4& nw, float (&f)[8]) {
    float w[8];
    load8(kept(v), true, 0, f);
    unpack8_bf16(nw, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = (f[q] * rn) * w[q];
  };
  auto write8 = [&](int v, const uint4& nw) {  // (whole warps: a group's maximum is a shuffle)
    float f[8], m = 0.f;
    if (on && v < nv) {
      next8(v, nw, f);
#pragma unroll
      for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(f[q]));
      if (tail.xhat) store8_bf16(tail.xhat + (size_t)t * H + v * 8, f);
    }
    if (tail.xq && tail.q_group) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = m > 0.f ? __fdiv_rn(m, 448.0f) : 1.0f;
      if (on && v < nv) {
        *reinterpret_cast<uint2*>(tail.xq + (size_t)t * H + v * 8) = tail_e4m3x8(f, s);
        if ((v & 15) == 0) tail.xscale[(size_t)t * (H >> 7) + (v >> 4)] = s;
      }
    }
    amax = fmaxf(amax, m);
  };
#pragma unroll
  for (int i = 0; i < kPre; ++i) write8(sub + i * ntr, pre_nw[i]);
#pragma unroll 2
  for (int v0 = kPre * ntr; v0 < nv; v0 += ntr) {
    uint4 nw = make_uint4(0u, 0u, 0u, 0u);
    if (v0 + sub < nv) nw = reinterpret_cast<const uint4*>(tail.next_w)[v0 + sub];
    write8(v0 + sub, nw);
  }
  if (tail.xq && !tail.q_group) {
    amax = row_reduce(amax, true);
    const float s = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (on) {
      for (int v = sub; v < nv; v += ntr) {
        float f[8];
        next8(v, reinterpret_cast<const uint4*>(tail.next_w)[v], f);
        *reinterpret_cast<uint2*>(tail.xq + (size_t)t * H + v * 8) = tail_e4m3x8(f, s);
      }
      if (sub == 0) tail.xscale[t] = s;
    }
  }
}

}  // namespace

namespace {
struct LayerWs {
  size_t hi, lo, ssq, part, ctr, act_hi, act_lo, f, total;
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
  w.part = take((size_t)kLayerChunks * t * E * 4);
  w.ctr = take(16);
  w.act_hi = take(t * k * I * 2);
  w.act_lo = take(t * k * I * 2);
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
  p.hi = reinterpret_cast<bf16*>(ws + w.hi);
  p.lo = reinterpret_cast<bf16*>(ws + w.lo);
  p.act_hi = reinterpret_cast<bf16*>(ws + w.act_hi);
  p.act_lo = reinterpret_cast<bf16*>(ws + w.act_lo);
  p.ssq = reinterpret_cast<float*>(ws + w.ssq);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.f = reinterpret_cast<float*>(ws + w.f);
  p.ctr = reinterpret_cast<int*>(ws + w.ctr);
  p.status = status;
  const int rows = (a.H / 8 + kLayerChunks - 1) / kLayerChunks * 8;
  cudaError_t e =
      launch_kernel(layer_route_kernel, dim3(kLayerChunks, a.router_w ? (a.E + 31) / 32 : 1),
                    dim3(32 * kRouteWarps), a.router_w ? (size_t)rows * kLayerMaxT * 4 : 0, st, p);
  if (e != cudaSuccess) return e;
  auto kern = a.fp8 ? layer_experts_kernel<true> : layer_experts_kernel<false>;
  const int smem = a.fp8 ? Ring<true>::kBytes : Ring<false>::kBytes;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(sms), dim3(kThreadsL), smem, st, p, tail ? *tail : TailP{},
                       tail ? 1 : 0);
}

}  // namespace moe
