// Host-side launch functions of the operators around the experts' products:
// weighted return of expert rows, layer norm, dense product, and their
// gradients (internal to libmoeffn).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ------------------------------------------------------------------ rows.cu --
constexpr int kRowsMaxH = 32768;

// out[t] = residual[t] + sum_j w[t, j] y[row_of_pair[t, j]]; w NULL: 1.
struct UnpermuteArgs {
  const void* y;
  const int32_t* row_of_pair;
  const float* w;
  const void* residual;
  void* out;
  int T, k, H;
  bool y_f32, res_f32, out_f32;
};
cudaError_t launch_unpermute(const UnpermuteArgs& a, int* status, cudaStream_t st);

struct UnpermuteGradArgs {
  const void* dout;
  const void* y;
  const int32_t* row_of_pair;
  const float* w;
  const int32_t* ids;
  void* dy;        // or NULL
  float* dw;       // or NULL
  float* dlogits;  // or NULL
  int T, k, H, E;
  bool dout_f32, y_f32;
};
cudaError_t launch_unpermute_grad(const UnpermuteGradArgs& a, int sms, int* status, cudaStream_t st);

// ------------------------------------------------------------------ norm.cu --
constexpr int kNormMaxH = 16384;

struct LayerNormArgs {
  const void* x;
  const void* w;
  const void* b;  // or NULL
  void* y;
  float* mean;    // or NULL
  float* rstd;    // or NULL
  int T, H;
  float eps;
  bool x_f32, y_f32, w_f32;
};
cudaError_t launch_layernorm(const LayerNormArgs& a, int sms, int* status, cudaStream_t st);

struct NormGradArgs {
  const void* dy;
  const void* x;
  const void* w;
  const float* mean;  // NULL: rms_norm, statistics from x
  const float* rstd;
  const void* dres;   // or NULL, x's type
  void* dx;
  float* dw;
  float* db;          // or NULL
  void* workspace;
  int T, H;
  float eps;
  bool x_f32, dy_f32, w_f32;
};
size_t norm_grad_workspace_bytes(int T, int H);
cudaError_t launch_norm_grad(const NormGradArgs& a, int sms, int* status, cudaStream_t st);

// ---------------------------------------------------------------- linear.cu --
enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// The form of a product: chosen by its size, or the one that MOE_LINEAR_FORM names.
enum LinearForm { kFormAuto = 0, kFormToken, kFormSplit, kFormPair };
// What `name` (NULL and "": kFormAuto) says; false if no form has that name.
bool linear_form(const char* name, LinearForm* form);

// One product D[q, p] = sum_k a[p, k] b[q, k] with p the contiguous index of the
// output, and its epilogue out = residual + act(D + bias).  a_mn: a is stored [K, P]
// instead of [P, K]; b_mn likewise.
struct ProductArgs {
  const void* a;
  const void* b;
  bool a_mn, b_mn;
  int64_t P, Q, K;
  const void* bias;      // [P] or NULL
  const void* residual;  // [Q, P] or NULL
  void* pre;             // bf16 [Q, P] or NULL: D + bias
  void* out;             // [Q, P]
  int act;
  bool bias_f32, res_f32, out_f32;
  LinearForm form;  // kFormToken: Q = 1, a and b K-major
};
cudaError_t launch_product(const ProductArgs& a, int sms, int* status, cudaStream_t st);

// dpre = dout * act'(pre) in bf16 (or NULL: not stored) and db = its column sums, before the
// rounding (or NULL).
constexpr int kActGradRows = 256;  // partial sums per column at most
struct ActGradArgs {
  const void* dout;
  const void* pre;  // bf16, NULL without activation
  void* dpre;
  float* db;
  float* part;      // [kActGradRows, N]
  int64_t M, N;
  int act;
  bool dout_f32;
};
cudaError_t launch_act_grad(const ActGradArgs& a, int sms, cudaStream_t st);

}  // namespace moe
