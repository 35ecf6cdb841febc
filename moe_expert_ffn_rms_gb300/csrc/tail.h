// Host-side launch functions of the fused block tail and the few-token layer
// (internal to libmoeffn).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "block_tail.cuh"

namespace moe {

// moe_combine_norm; H <= kTailMaxH.
constexpr int kTailMaxH = 32768;
constexpr int kStreamSmem = 226 << 10;  // shared memory per SM the streaming form plans with
constexpr int kStreamStatic = 2048;     // of which a CTA's static part and the runtime's reserve
constexpr int kStreamStages = 8;        // stages per CTA at most
constexpr int kStreamCtas = 16;         // CTAs per SM at most
cudaError_t launch_combine_norm(const void* y, bool y_f32, bool pair_order,
                                const int32_t* row_of_pair, int T, int k, int H, const TailP& p,
                                int* status, int sms, cudaStream_t st);

// moe_layer_forward: the whole block for T <= kLayerMaxT tokens (layer.cu).
constexpr int kLayerMaxT = 8;
constexpr int kLayerChunks = 16;  // K chunks of the router's partial sums
constexpr int kLayerMaxH = 16384;

struct LayerArgs {
  const void* x;
  const void* norm_w;
  const float* router_w;  // one of router_w, logits, ids_in (with tw_in)
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
  void* out;
  void* workspace;
  int T, H, E, I, k;
  bool fp8, block_scales;
  float eps;
};

size_t layer_workspace_bytes(int T, int H, int E, int I, int k, bool fp8);
cudaError_t launch_layer(const LayerArgs& a, const TailP* tail, int sms, int* status, cudaStream_t st);

}  // namespace moe
