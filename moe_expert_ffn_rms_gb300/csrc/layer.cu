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
// bf16; accumulation is fp32.  A warp reads its own weights: each lane copies
// exactly the 16-byte pieces it will feed to its MMAs into its own part of
// shared memory (cp.async, kStages steps ahead) and reads them back, so the
// stream needs no barrier, and the first W2 pieces are already on their way
// while the CTA waits for the other CTAs' FC1 tiles.  The order of the K
// elements inside a piece is the same for both operands and therefore free.
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
constexpr int kStages = 6;                      // steps in flight per warp
constexpr int kStepBytes = 4096;                // per warp: 2 tiles x 2 row halves x 2 K blocks x 512 B
constexpr int kRingBytes = kWarps * kStages * kStepBytes;
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
__global__ void __launch_bounds__(kThreadsL) layer_route_kernel(const LayerP p) {
  extern __shared__ __align__(16) float xw[];  // [rows of the chunk][8 tokens]
  __shared__ float red[kWarps][kLayerMaxT][32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x, nb = p.H >> 3;
  const int b0 = (int)((int64_t)c * nb / kLayerChunks), b1 = (int)((int64_t)(c + 1) * nb / kLayerChunks);
  const int k0 = b0 * 8, rows = (b1 - b0) * 8;
  if (c == 0 && blockIdx.y == 0 && tid < 4) p.ctr[tid] = 0;
  const int e = blockIdx.y * 32 + lane;
  const float* wr = p.router_w ? p.router_w + (size_t)k0 * p.E + e : nullptr;
  constexpr int U = 8;
  float wv[U];
  if (wr) {  // the first rows of W_r are on their way while x is prepared
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = warp + kWarps * u;
      wv[u] = (r < rows && e < p.E) ? wr[(size_t)r * p.E] : 0.f;
    }
  }
  // warp t: token t
  float ss = 0.f;
  for (int v = lane; v < b1 - b0; v += 32) {
    float a[8], hi[8], lo[8];
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
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] = 0.f;
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
  if (!wr) return;
  __syncthreads();
  float acc[kLayerMaxT];
#pragma unroll
  for (int t = 0; t < kLayerMaxT; ++t) acc[t] = 0.f;
  for (int r0 = warp; r0 < rows; r0 += kWarps * U) {
    float nx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + kWarps * (U + u);
      nx[u] = (r < rows && e < p.E) ? wr[(size_t)r * p.E] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + kWarps * u;
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
      wv[u] = nx[u];
    }
  }
#pragma unroll
  for (int t = 0; t < kLayerMaxT; ++t) red[warp][t][lane] = acc[t];
  __syncthreads();
  if (warp < p.T && e < p.E) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w][warp][lane];
    p.part[((size_t)c * p.T + warp) * p.E + e] = s;
  }
}

// ------------------------------------------------------------------ launch 2 --
MOE_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most n of the newest groups are in flight.
MOE_DEV void cp_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}

MOE_DEV void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  asm volatile(
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

// A lane's activations for one step: two K blocks of EPC elements in two bf16
// terms, for the token of the lane's column.
template <int EPC>
struct StepB {
  uint4 hi[2][EPC / 8], lo[2][EPC / 8];
  float s[2][2];  // FP8: weight scales of the lane's four rows
};

struct LayerSmem {
  int32_t ids[kLayerMaxT][kMaxTopK];
  float w[kLayerMaxT][kMaxTopK];
  float r[kLayerMaxT];
  int expert[kMaxPairs];
  unsigned mask[kMaxPairs];
  int pair[kMaxPairs][kLayerMaxT];
  float wt[kMaxPairs][kLayerMaxT];
  int warp_cnt[kWarps];
  int claim[4];
  int n_act;
  int flag;
  float sum[kWarps];
};

template <int PER>
MOE_DEV void layer_topk(const LayerP& p, int t, int lane, float r, LayerSmem* sm) {
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    v[i] = -INFINITY;
    if (e < p.E) {
      float z = 0.f;
      if (p.logits) {
        z = p.logits[(size_t)t * p.E + e];
      } else {
#pragma unroll
        for (int c = 0; c < kLayerChunks; ++c) z += __ldcg(&p.part[((size_t)c * p.T + t) * p.E + e]);
        z *= r;
      }
      v[i] = p.bias ? z + p.bias[e] : z;
    }
  }
  warp_topk<PER>(v, p.E, p.k, lane, sm->ids[t], sm->w[t]);
}

// FP8: E4M3 weights with scales, one per (row >> rs, K step * ks).
template <bool FP8>
__global__ void __launch_bounds__(kThreadsL, 1) layer_experts_kernel(const LayerP p, const TailP tail,
                                                                     int has_tail) {
  constexpr int EB = FP8 ? 1 : 2;   // bytes per weight
  constexpr int EPC = 16 / EB;      // weights per 16-byte piece
  constexpr int KE = 64 / EB;       // K elements of a K block (64 bytes of a row)
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ LayerSmem sm;
  __shared__ __align__(16) float red[2][kRedFloats];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tq = lane & 3;  // MMA fragment row / column group, K group
  const int T = p.T, H = p.H, E = p.E, I = p.I, k = p.k;
  pdl_trigger();
  pdl_wait();

  // ---- routing (every CTA by itself; warp t: token t)
  if (tid == 0) {
    sm.claim[0] = atomicAdd(&p.ctr[0], 1);
    sm.claim[1] = atomicAdd(&p.ctr[0], 1);
    sm.n_act = 0;
  }
  if (warp < T) {
    float ss = lane < kLayerChunks ? __ldcg(&p.ssq[lane * kLayerMaxT + warp]) : 0.f;
    const float r = 1.0f / sqrtf(warp_sum(ss) / (float)H + p.eps);
    if (lane == 0) sm.r[warp] = r;
    if (p.ids_in) {
      if (lane < k) {
        sm.ids[warp][lane] = p.ids_in[warp * k + lane];
        sm.w[warp][lane] = p.tw_in[warp * k + lane];
      }
    } else if (E <= 32) {
      layer_topk<1>(p, warp, lane, r, &sm);
    } else if (E <= 64) {
      layer_topk<2>(p, warp, lane, r, &sm);
    } else if (E <= 128) {
      layer_topk<4>(p, warp, lane, r, &sm);
    } else {
      layer_topk<8>(p, warp, lane, r, &sm);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid < T * k) {
    const int id = sm.ids[tid / k][tid % k];
    if (p.ids_out) p.ids_out[tid] = id;
    if (p.tw_out) p.tw_out[tid] = sm.w[tid / k][tid % k];
    if (id < 0 || id >= E) flag_status(p.status, MOE_ERR_INVALID_ARG);
  }
  // active experts in ascending order (thread e: expert e; E <= 256)
  {
    unsigned mask = 0;
    for (int i = 0; i < T * k; ++i)
      if (tid < E && sm.ids[i / k][i % k] == tid) mask |= 1u << (i / k);
    const unsigned act = __ballot_sync(0xffffffffu, mask != 0);
    if (lane == 0) sm.warp_cnt[warp] = __popc(act);
    __syncthreads();
    if (mask) {
      int at = __popc(act & ((1u << lane) - 1));
      for (int w = 0; w < warp; ++w) at += sm.warp_cnt[w];
      sm.expert[at] = tid;
      sm.mask[at] = mask;
      for (int t = 0; t < kLayerMaxT; ++t) {
        int pr = -1;
        float w = 0.f;
        if ((mask >> t) & 1u)
          for (int j = 0; j < k; ++j)
            if (sm.ids[t][j] == tid) {  // (an expert given twice counts with both weights)
              if (pr < 0) pr = t * k + j;
              w += sm.w[t][j];
            }
        sm.pair[at][t] = pr;
        sm.wt[at][t] = w;
      }
    }
    if (tid == 0) {
      int n = 0;
      for (int w = 0; w < kWarps; ++w) n += sm.warp_cnt[w];
      sm.n_act = n;
    }
    __syncthreads();
  }
  const int n_act = sm.n_act;

  // ---- work: FC1 row tiles (8 gate + 8 up rows) in claims of two, the last
  // ones (one per CTA) single; FC2 output rows [n0, n1) in units of 32
  const int tiles_e = I >> 3;
  const int tiles = n_act * tiles_e;
  const int singles = min(tiles, (int)gridDim.x & ~1);
  const int pairs = (tiles - singles) >> 1;  // tiles and singles are even
  const int claims = pairs + singles;
  const int n0 = (int)((int64_t)blockIdx.x * H / gridDim.x);
  const int n1 = (int)((int64_t)(blockIdx.x + 1) * H / gridDim.x);
  const size_t rb1 = (size_t)H * EB, rb2 = (size_t)I * EB;  // bytes of a weight row
  const int S1 = (int)((rb1 + 127) >> 7), S2 = (int)((rb2 + 127) >> 7);  // 128-byte steps of a row
  const int kb1 = (int)(rb1 >> 6), kb2 = (int)(rb2 >> 6);                // 64-byte K blocks
  const unsigned char* w13 = static_cast<const unsigned char*>(p.w13);
  const unsigned char* w2 = static_cast<const unsigned char*>(p.w2);

  unsigned char* ring = ring_all + warp * (kStages * kStepBytes);
  const uint32_t ring_u = ptx::smem_u32(ring) + lane * 16;

  // ---- producer: the warp's steps in the order it will use them
  int pn = 0;           // FC1 claim being produced (index into this CTA's claims)
  int p_step = warp;    // next step of it
  int pu = 0, pa = 0;   // FC2 unit and active expert being produced
  bool p_fc2 = false;
  int known = 1;        // newest claim index published to this warp
  int issued = 0, used = 0;
  auto claim_tile = [&](int c) { return c < pairs ? 2 * c : c + pairs; };

  // Copies the next step if it is known; false when nothing can be copied yet.
  auto produce = [&]() -> bool {
    while (!p_fc2) {
      if (pn > known) return false;
      if (sm.claim[pn & 3] >= claims) {
        p_fc2 = true;
        p_step = warp;
      } else if (p_step >= S1) {
        ++pn;
        p_step = warp;
      } else {
        break;
      }
    }
    const unsigned char* src;
    size_t ts, hs;       // byte strides of the second tile and of a tile's lower 8 rows
    unsigned ok;         // bit 2*tile + half: this lane's row is wanted
    bool two;            // the step's second K block exists
    if (!p_fc2) {
      const int c = sm.claim[pn & 3];
      const int tile = claim_tile(c);
      const int a = tile / tiles_e;
      const int row = (tile - a * tiles_e) * 8 + g;
      src = w13 + ((size_t)sm.expert[a] * 2 * I + row) * rb1;
      ts = 8 * rb1;
      hs = (size_t)I * rb1;
      ok = c < pairs ? 15u : 3u;
      two = 2 * p_step + 1 < kb1;
    } else {
      while (p_step >= S2) {
        p_step -= S2;
        ++pa;
      }
      while (pa >= n_act) {  // next unit of output rows
        if (n_act == 0 || n0 + 32 * (pu + 1) >= n1) {
          pa = n_act;
          return false;
        }
        ++pu;
        pa = 0;
        p_step = warp;
        while (p_step >= S2) {
          p_step -= S2;
          ++pa;
        }
      }
      const int row = n0 + 32 * pu + g;
      src = w2 + ((size_t)sm.expert[pa] * H + row) * rb2;
      ts = 16 * rb2;
      hs = 8 * rb2;
      ok = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) ok |= (row + 8 * i < n1 ? 1u : 0u) << i;
      two = 2 * p_step + 1 < kb2;
    }
    src += (size_t)p_step * 128 + tq * 16;
    const uint32_t dst = ring_u + (issued % kStages) * kStepBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((ok >> i) & 1u) {
        const unsigned char* s = src + (i >> 1) * ts + (i & 1) * hs;
        cp_async16(dst + (2 * i) * 512, s);
        if (two) cp_async16(dst + (2 * i + 1) * 512, s + 64);
      }
    }
    cp_commit();
    ++issued;
    p_step += kWarps;
    return true;
  };
  auto top_up = [&]() {
    while (issued - used < kStages && produce()) {
    }
  };

  // One step: acc[tile] += weights of the step * activations b.
  auto multiply = [&](float (&acc)[2][4], const StepB<EPC>& b, bool second_tile, bool two) {
    cp_wait(issued - used - 1);
    const uint4* sp = reinterpret_cast<const uint4*>(ring + (used % kStages) * kStepBytes) + lane;
#pragma unroll
    for (int tl = 0; tl < 2; ++tl) {
      if (tl && !second_tile) break;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb && !two) break;
        const uint4 u0 = sp[((tl * 2 + 0) * 2 + kb) * 32], u1 = sp[((tl * 2 + 1) * 2 + kb) * 32];
        const uint32_t q0[4] = {u0.x, u0.y, u0.z, u0.w}, q1[4] = {u1.x, u1.y, u1.z, u1.w};
        if constexpr (!FP8) {
          const uint4 h = b.hi[kb][0], l = b.lo[kb][0];
          mma_16816(acc[tl], q0[0], q1[0], q0[1], q1[1], h.x, h.y);
          mma_16816(acc[tl], q0[0], q1[0], q0[1], q1[1], l.x, l.y);
          mma_16816(acc[tl], q0[2], q1[2], q0[3], q1[3], h.z, h.w);
          mma_16816(acc[tl], q0[2], q1[2], q0[3], q1[3], l.z, l.w);
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_bf16(q0[m], a0, a2);
            e4m3x4_bf16(q1[m], a1, a3);
            const uint4 h = b.hi[kb][m >> 1], l = b.lo[kb][m >> 1];
            mma_16816(acc[tl], a0, a1, a2, a3, (m & 1) ? h.z : h.x, (m & 1) ? h.w : h.y);
            mma_16816(acc[tl], a0, a1, a2, a3, (m & 1) ? l.z : l.x, (m & 1) ? l.w : l.y);
          }
        }
      }
    }
    ++used;
  };
  // Activations of K blocks 2*step, 2*step + 1 from row `row` (negative: zeros).
  auto load_b = [&](StepB<EPC>& b, const bf16* hi, const bf16* lo, int64_t row, int K, int step, int nkb) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int q = 0; q < EPC / 8; ++q) {
        b.hi[kb][q] = b.lo[kb][q] = make_uint4(0u, 0u, 0u, 0u);
        if (row >= 0 && 2 * step + kb < nkb) {
          const size_t at = (size_t)row * K + (size_t)(2 * step + kb) * KE + tq * EPC + q * 8;
          b.hi[kb][q] = __ldcg(reinterpret_cast<const uint4*>(hi + at));
          b.lo[kb][q] = __ldcg(reinterpret_cast<const uint4*>(lo + at));
        }
      }
    }
  };
  // FP8 scales of the lane's rows row, row + hs (and a tile further, + ts) at a step.
  auto load_s = [&](StepB<EPC>& b, const float* s, int e, int N, int K, int row, int ts, int hs, unsigned ok,
                    int step) {
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rw = row + (i >> 1) * ts + (i & 1) * hs;
        b.s[i >> 1][i & 1] = 0.f;
        if ((ok >> i) & 1u)
          b.s[i >> 1][i & 1] = p.block_scales
                                   ? s[((size_t)e * (N >> 7) + (rw >> 7)) * (K >> 7) + step]
                                   : s[(size_t)e * N + rw];
      }
    }
  };
  // tot += scale * acc for the tokens in mask; a column outside it adds nothing
  // (not 0 times a weight that may not be finite).
  auto fold = [&](float (&tot)[2][4], const float (&acc)[2][4], const StepB<EPC>& b, unsigned mask) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((mask >> (2 * tq + (i & 1))) & 1u)
          tot[tl][i] = FP8 ? fmaf(b.s[tl][i >> 1], acc[tl][i], tot[tl][i]) : tot[tl][i] + acc[tl][i];
  };
  auto store_red = [&](float* rd, const float (&tot)[2][4]) {
#pragma unroll
    for (int tl = 0; tl < 2; ++tl) {
      float* d = rd + ((warp * 2 + tl) * 16 + g) * 8 + 2 * tq;
      *reinterpret_cast<float2*>(d) = make_float2(tot[tl][0], tot[tl][1]);
      *reinterpret_cast<float2*>(d + 64) = make_float2(tot[tl][2], tot[tl][3]);
    }
  };

  top_up();
  int buf = 0;
  int my_tiles = 0;

  // ---- FC1
  for (int n = 0;; ++n) {
    const int c = sm.claim[n & 3];
    if (c >= claims) break;
    int next_claim = claims;
    if (tid == 0) next_claim = atomicAdd(&p.ctr[0], 1);  // used two claims from here
    const int tile = claim_tile(c);
    const int nt = c < pairs ? 2 : 1;
    const int a = tile / tiles_e;
    const int i0 = (tile - a * tiles_e) * 8;
    const int e = sm.expert[a];
    const unsigned mask = sm.mask[a];
    const int64_t brow = ((mask >> g) & 1u) ? g : -1;
    float tot[2][4] = {};
    StepB<EPC> b;
    if (warp < S1) {
      load_b(b, p.hi, p.lo, brow, H, warp, kb1);
      load_s(b, p.s13, e, 2 * I, H, i0 + g, 8, I, nt == 2 ? 15u : 3u, warp);
    }
    for (int step = warp; step < S1; step += kWarps) {
      StepB<EPC> nb;
      if (step + kWarps < S1) {
        load_b(nb, p.hi, p.lo, brow, H, step + kWarps, kb1);
        load_s(nb, p.s13, e, 2 * I, H, i0 + g, 8, I, nt == 2 ? 15u : 3u, step + kWarps);
      }
      if constexpr (FP8) {
        float acc[2][4] = {};
        multiply(acc, b, nt == 2, 2 * step + 1 < kb1);
        fold(tot, acc, b, mask);
      } else {
        multiply(tot, b, nt == 2, 2 * step + 1 < kb1);
      }
      top_up();
      b = nb;
    }
    store_red(red[buf], tot);
    if (tid == 0) sm.claim[(n + 2) & 3] = next_claim;
    __syncthreads();
    known = n + 2;
    // 16 consecutive threads: the 16 intermediate columns of one token
    if (tid < 128) {
      const int t = tid >> 4, il = tid & 15;
      if (((mask >> t) & 1u) && (il >> 3) < nt) {
        const float* s = red[buf] + ((il >> 3) * 16 + (il & 7)) * 8 + t;
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          gate += s[w * 256];
          up += s[w * 256 + 64];
        }
        const float r = sm.r[t];
        // the routing weight goes into the intermediate, so FC2 adds the
        // token's experts without a factor
        const float v = silu_f(gate * r) * (up * r) * sm.wt[a][t];
        const float hi = bf16_round_f(v);
        const size_t at = (size_t)sm.pair[a][t] * I + i0 + il;
        p.act_hi[at] = __float2bfloat16_rn(hi);
        p.act_lo[at] = __float2bfloat16_rn(v - hi);
      }
    }
    my_tiles += nt;
    buf ^= 1;
    top_up();
  }
  // ---- all FC1 tiles done (each CTA's writes are visible before its count)
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

  // ---- FC2: this CTA's output rows over all active experts
  for (int u = 0; n0 + 32 * u < n1; ++u) {
    const int row0 = n0 + 32 * u;
    unsigned ok = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) ok |= (row0 + g + 8 * i < n1 ? 1u : 0u) << i;
    const bool second = row0 + 16 < n1;
    float tot[2][4] = {};
    StepB<EPC> b;
    int a = 0, step = warp;
    while (step >= S2) {
      step -= S2;
      ++a;
    }
    if (a < n_act) {
      load_b(b, p.act_hi, p.act_lo, sm.pair[a][g], I, step, kb2);
      load_s(b, p.s2, sm.expert[a], H, I, row0 + g, 16, 8, ok, step);
    }
    while (a < n_act) {
      int na = a, ns = step + kWarps;
      while (ns >= S2) {
        ns -= S2;
        ++na;
      }
      StepB<EPC> nb;
      if (na < n_act) {
        load_b(nb, p.act_hi, p.act_lo, sm.pair[na][g], I, ns, kb2);
        load_s(nb, p.s2, sm.expert[na], H, I, row0 + g, 16, 8, ok, ns);
      }
      float acc[2][4] = {};
      multiply(acc, b, second, 2 * step + 1 < kb2);
      fold(tot, acc, b, sm.mask[a]);
      top_up();
      b = nb;
      a = na;
      step = ns;
    }
    store_red(red[buf], tot);
    __syncthreads();
    const int row = tid & 31, t = tid >> 5;
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

  // ---- tail: the CTA that finishes last takes all rows
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    sm.flag = atomicAdd(&p.ctr[2], 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!sm.flag) return;
  // 256 / Tp threads per row (Tp: T rounded up to a power of two)
  const int tp = T <= 1 ? 1 : (T <= 2 ? 2 : (T <= 4 ? 4 : 8));
  const int ntr = kThreadsL / tp, wpr = kWarps / tp;
  const int t = tid / ntr, sub = tid - t * ntr;
  const bool on = t < T;
  const int nv = H >> 3;
  auto row_reduce = [&](float v, bool mx) {
    v = mx ? warp_max(v) : warp_sum(v);
    if (lane == 0) sm.sum[warp] = v;
    __syncthreads();
    v = sm.sum[t * wpr];
    for (int w = 1; w < wpr; ++w) v = mx ? fmaxf(v, sm.sum[t * wpr + w]) : v + sm.sum[t * wpr + w];
    __syncthreads();
    return v;
  };
  auto load_f = [&](int c, float (&v)[8]) {
    const float4* s = reinterpret_cast<const float4*>(p.f + (size_t)t * H + c);
    const float4 a = __ldcg(s), b = __ldcg(s + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  };
  float r = 1.f;
  if (tail.post_w) {
    float ss = 0.f;
    if (on) {
#pragma unroll 4
      for (int v = sub; v < nv; v += ntr) {
        float f[8];
        load_f(v * 8, f);
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(f[q], f[q], ss);
      }
    }
    r = 1.0f / sqrtf(row_reduce(ss, false) / (float)H + tail.post_eps);
  }
  const int grow = on ? tail_gate_row(tail, t, sub == 0 ? p.status : nullptr) : 0;
  const float factor = on ? tail_row_factor(tail, grow) : 0.f;
  float ss = 0.f;
  if (on) {
#pragma unroll 2
    for (int v = sub; v < nv; v += ntr) {
      float f[8], h[8], res[8];
      load_f(v * 8, f);
      if (tail.residual) {
        load8(tail.residual, tail.res_f32 != 0, (size_t)t * H + v * 8, res);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) res[q] = 0.f;
      }
      tail_h8(tail, H, v * 8, f, r, grow, factor, res, h);
      store8(tail.out, tail.out_f32 != 0, (size_t)t * H + v * 8, h);
      if (tail.next_w) {
        float4* d = reinterpret_cast<float4*>(p.f + (size_t)t * H + v * 8);  // read back by this thread
        __stcg(d, make_float4(h[0], h[1], h[2], h[3]));
        __stcg(d + 1, make_float4(h[4], h[5], h[6], h[7]));
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(h[q], h[q], ss);
      }
    }
  }
  if (!tail.next_w) return;
  r = 1.0f / sqrtf(row_reduce(ss, false) / (float)H + tail.next_eps);
  float amax = 0.f;
  auto next8 = [&](int v, float (&f)[8]) {
    float w[8];
    load_f(v * 8, f);
    load8(tail.next_w, false, v * 8, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = (f[q] * r) * w[q];
  };
  for (int v0 = 0; v0 < nv; v0 += ntr) {
    const int v = v0 + sub;
    float f[8], m = 0.f;
    if (on && v < nv) {
      next8(v, f);
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
  }
  if (tail.xq && !tail.q_group) {
    amax = row_reduce(amax, true);
    const float s = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (on) {
      for (int v = sub; v < nv; v += ntr) {
        float f[8];
        next8(v, f);
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
                    dim3(kThreadsL), a.router_w ? (size_t)rows * kLayerMaxT * 4 : 0, st, p);
  if (e != cudaSuccess) return e;
  auto kern = a.fp8 ? layer_experts_kernel<true> : layer_experts_kernel<false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(sms), dim3(kThreadsL), kRingBytes, st, p, tail ? *tail : TailP{},
                       tail ? 1 : 0);
}

}  // namespace moe
