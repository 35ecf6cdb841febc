// extern "C" entry points of the operators around the experts' products:
// argument checks and launches.
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>

#include "api_internal.h"
#include "common.cuh"
#include "train.h"

namespace {

moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return moe::api_fail(s, buf);
}

#define MOE_REQ(cond, code, ...) \
  do {                           \
    if (!(cond)) return fail(code, __VA_ARGS__); \
  } while (0)

#define MOE_CUDA(call, what)                                                     \
  do {                                                                           \
    cudaError_t _e = (call);                                                     \
    if (_e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(_e)); \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

moe_status check_rows(int T, int k, int H) {
  MOE_REQ(T >= 0 && k > 0 && k <= kMaxTopK && H > 0 && H % 8 == 0 && H <= moe::kRowsMaxH &&
              (int64_t)T * k <= (1 << 24),
          MOE_ERR_UNSUPPORTED_SHAPE, "T=%d k=%d H=%d (k <= %d, H %% 8 == 0, H <= %d, T*k <= 2^24)", T, k,
          H, kMaxTopK, moe::kRowsMaxH);
  return MOE_OK;
}

moe_status unpermute(const void* y, int y_bf16, const int32_t* row_of_pair, const float* topk_w, int T,
                     int k, int H, const void* residual, int residual_f32, void* out, int out_f32,
                     moe_stream_t stream) {
  moe_status rc = check_rows(T, k, H);
  if (rc != MOE_OK || T == 0) return rc;
  MOE_REQ(y && row_of_pair && out, MOE_ERR_INVALID_ARG, "the rows, row_of_pair and the output must be non-NULL");
  MOE_REQ(aligned(y, 16) && aligned(residual, 16) && aligned(out, 16) && aligned(row_of_pair, 4) &&
              aligned(topk_w, 4),
          MOE_ERR_INVALID_ARG, "misaligned pointer");
  MOE_REQ(residual != out || (residual_f32 != 0) == (out_f32 != 0), MOE_ERR_INVALID_ARG,
          "the row that is added may be the output only when both have one type");
  int sms = 0, *status = nullptr;
  if ((rc = moe::api_device(&sms, &status)) != MOE_OK) return rc;
  moe::UnpermuteArgs a{};
  a.y = y;
  a.row_of_pair = row_of_pair;
  a.w = topk_w;
  a.residual = residual;
  a.out = out;
  a.T = T;
  a.k = k;
  a.H = H;
  a.y_f32 = y_bf16 == 0;
  a.res_f32 = residual_f32 != 0;
  a.out_f32 = out_f32 != 0;
  MOE_CUDA(moe::launch_unpermute(a, status, (cudaStream_t)stream), "unpermute launch");
  return MOE_OK;
}

moe_status check_norm(int T, int H) {
  MOE_REQ(T >= 0 && H > 0 && H % 8 == 0 && H <= moe::kNormMaxH, MOE_ERR_UNSUPPORTED_SHAPE,
          "T=%d H=%d (H %% 8 == 0, H <= %d)", T, H, moe::kNormMaxH);
  return MOE_OK;
}

moe_status norm_grad(moe::NormGradArgs& a, size_t workspace_bytes, moe_stream_t stream) {
  moe_status rc = check_norm(a.T, a.H);
  if (rc != MOE_OK) return rc;
  MOE_REQ(a.dw && aligned(a.dw, 4) && aligned(a.db, 4), MOE_ERR_INVALID_ARG,
          "dw must be non-NULL, dw and db 4-byte aligned");
  MOE_REQ(a.eps >= 0.f, MOE_ERR_INVALID_ARG, "eps < 0");
  if (a.T > 0) {
    MOE_REQ(a.dy && a.x && a.w && a.dx, MOE_ERR_INVALID_ARG, "dy, x, w and dx must be non-NULL");
    MOE_REQ(aligned(a.dy, 16) && aligned(a.x, 16) && aligned(a.w, 16) && aligned(a.dx, 16) &&
                aligned(a.dres, 16) && aligned(a.mean, 4) && aligned(a.rstd, 4),
            MOE_ERR_INVALID_ARG, "misaligned pointer");
    MOE_REQ(a.dx != a.dy || a.x_f32 == a.dy_f32, MOE_ERR_INVALID_ARG, "dx may be dy only when both have one type");
    const size_t need = moe::norm_grad_workspace_bytes(a.T, a.H);
    MOE_REQ(workspace_bytes >= need && a.workspace, MOE_ERR_WORKSPACE_TOO_SMALL,
            "norm backward workspace %zu < %zu bytes", workspace_bytes, need);
    MOE_REQ(aligned(a.workspace, 256), MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  int sms = 0, *status = nullptr;
  if ((rc = moe::api_device(&sms, &status)) != MOE_OK) return rc;
  MOE_CUDA(moe::launch_norm_grad(a, sms, status, (cudaStream_t)stream), "norm backward launch");
  return MOE_OK;
}

constexpr int kLinearMaxM = 1 << 23, kLinearMaxNK = 1 << 20;

moe_status check_linear(int M, int N, int K, int act) {
  MOE_REQ(M >= 0 && M <= kLinearMaxM && N > 0 && N <= kLinearMaxNK && N % 8 == 0 && K > 0 &&
              K <= kLinearMaxNK && K % 8 == 0,
          MOE_ERR_UNSUPPORTED_SHAPE, "M=%d N=%d K=%d (M <= 2^23; N, K multiples of 8, <= 2^20)", M, N, K);
  MOE_REQ(act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH, MOE_ERR_INVALID_ARG, "act=%d", act);
  return MOE_OK;
}

// MOE_LINEAR_FORM, read once per call.  `token`: whether the one-token kernel can run it.
moe_status read_form(bool token, moe::LinearForm* form) {
  const char* name = getenv("MOE_LINEAR_FORM");
  MOE_REQ(moe::linear_form(name, form), MOE_ERR_INVALID_ARG, "MOE_LINEAR_FORM=%.32s: token, split or pair", name);
  MOE_REQ(token || *form != moe::kFormToken, MOE_ERR_INVALID_ARG,
          "MOE_LINEAR_FORM=token: for moe_linear of one row alone");
  return MOE_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

extern "C" {

moe_status moe_unpermute(const void* y, int32_t y_bf16, const int32_t* row_of_pair,
                         const float* topk_w, int32_t T, int32_t k, int32_t H,
                         const void* residual, int32_t residual_f32, void* out, int32_t out_f32,
                         moe_stream_t stream) {
  return unpermute(y, y_bf16, row_of_pair, topk_w, T, k, H, residual, residual_f32, out, out_f32, stream);
}

moe_status moe_permute_backward(const void* dxp, int32_t dxp_bf16, const int32_t* row_of_pair,
                                int32_t T, int32_t k, int32_t H, const void* dres, int32_t dres_f32,
                                void* dx, int32_t dx_f32, moe_stream_t stream) {
  return unpermute(dxp, dxp_bf16, row_of_pair, nullptr, T, k, H, dres, dres_f32, dx, dx_f32, stream);
}

moe_status moe_unpermute_backward(const void* dout, int32_t dout_f32, const void* y, int32_t y_bf16,
                                  const int32_t* row_of_pair, const float* topk_w,
                                  const int32_t* ids, int32_t T, int32_t k, int32_t H, int32_t E,
                                  void* dy, float* dw, float* dlogits, moe_stream_t stream) {
  moe_status rc = check_rows(T, k, H);
  if (rc != MOE_OK) return rc;
  MOE_REQ(!dlogits || (E > 0 && E <= kMaxExperts), MOE_ERR_UNSUPPORTED_SHAPE, "E=%d (1 to %d)", E, kMaxExperts);
  if (T == 0) return MOE_OK;
  MOE_REQ(dout && row_of_pair && topk_w, MOE_ERR_INVALID_ARG, "dout, row_of_pair and topk_w must be non-NULL");
  MOE_REQ(dy || dw || dlogits, MOE_ERR_INVALID_ARG, "no output: give dy, dw or dlogits");
  MOE_REQ(y || !(dw || dlogits), MOE_ERR_INVALID_ARG, "dw and dlogits need y");
  MOE_REQ(ids || !dlogits, MOE_ERR_INVALID_ARG, "dlogits needs ids");
  MOE_REQ(aligned(dout, 16) && aligned(y, 16) && aligned(dy, 16) && aligned(row_of_pair, 4) &&
              aligned(topk_w, 4) && aligned(ids, 4) && aligned(dw, 4) && aligned(dlogits, 4),
          MOE_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0, *status = nullptr;
  if ((rc = moe::api_device(&sms, &status)) != MOE_OK) return rc;
  moe::UnpermuteGradArgs a{};
  a.dout = dout;
  a.y = y;
  a.row_of_pair = row_of_pair;
  a.w = topk_w;
  a.ids = ids;
  a.dy = dy;
  a.dw = dw;
  a.dlogits = dlogits;
  a.T = T;
  a.k = k;
  a.H = H;
  a.E = E;
  a.dout_f32 = dout_f32 != 0;
  a.y_f32 = y_bf16 == 0;
  MOE_CUDA(moe::launch_unpermute_grad(a, sms, status, (cudaStream_t)stream), "unpermute backward launch");
  return MOE_OK;
}

moe_status moe_layernorm(const void* x, int32_t x_f32, const void* w, const void* b, int32_t w_f32,
                         int32_t T, int32_t H, float eps, void* y, int32_t y_f32, float* mean,
                         float* rstd, moe_stream_t stream) {
  moe_status rc = check_norm(T, H);
  if (rc != MOE_OK) return rc;
  MOE_REQ(eps >= 0.f, MOE_ERR_INVALID_ARG, "eps < 0");
  MOE_REQ((mean == nullptr) == (rstd == nullptr), MOE_ERR_INVALID_ARG, "give both mean and rstd or neither");
  if (T == 0) return MOE_OK;
  MOE_REQ(x && w && y, MOE_ERR_INVALID_ARG, "x, w and y must be non-NULL");
  MOE_REQ(aligned(x, 16) && aligned(w, 16) && aligned(b, 16) && aligned(y, 16) && aligned(mean, 4) &&
              aligned(rstd, 4),
          MOE_ERR_INVALID_ARG, "misaligned pointer");
  MOE_REQ(x != y || (x_f32 != 0) == (y_f32 != 0), MOE_ERR_INVALID_ARG, "y may be x only when both have one type");
  int sms = 0, *status = nullptr;
  if ((rc = moe::api_device(&sms, &status)) != MOE_OK) return rc;
  moe::LayerNormArgs a{};
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.x_f32 = x_f32 != 0;
  a.y_f32 = y_f32 != 0;
  a.w_f32 = w_f32 != 0;
  MOE_CUDA(moe::launch_layernorm(a, sms, status, (cudaStream_t)stream), "layernorm launch");
  return MOE_OK;
}

size_t moe_norm_backward_workspace_size(int32_t T, int32_t H) {
  if (check_norm(T, H) != MOE_OK) return 0;
  const size_t n = moe::norm_grad_workspace_bytes(T, H);
  return n ? n : 256;  // (T = 0 needs none; 0 says that the shape is refused)
}

moe_status moe_layernorm_backward(const void* dy, int32_t dy_f32, const void* x, int32_t x_f32,
                                  const void* w, int32_t w_f32, const float* mean, const float* rstd,
                                  const void* dres, int32_t T, int32_t H, void* dx, float* dw,
                                  float* db, void* workspace, size_t workspace_bytes,
                                  moe_stream_t stream) {
  MOE_REQ(T <= 0 || (mean && rstd), MOE_ERR_INVALID_ARG, "mean and rstd must be non-NULL");
  moe::NormGradArgs a{};
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.mean = mean;
  a.rstd = rstd;
  a.dres = dres;
  a.dx = dx;
  a.dw = dw;
  a.db = db;
  a.workspace = workspace;
  a.T = T;
  a.H = H;
  a.x_f32 = x_f32 != 0;
  a.dy_f32 = dy_f32 != 0;
  a.w_f32 = w_f32 != 0;
  return norm_grad(a, workspace_bytes, stream);
}

moe_status moe_rmsnorm_backward(const void* dy, int32_t dy_f32, const void* x, int32_t x_f32,
                                const void* w, int32_t w_f32, float eps, const void* dres, int32_t T,
                                int32_t H, void* dx, float* dw, void* workspace,
                                size_t workspace_bytes, moe_stream_t stream) {
  moe::NormGradArgs a{};
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.dres = dres;
  a.dx = dx;
  a.dw = dw;
  a.workspace = workspace;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.x_f32 = x_f32 != 0;
  a.dy_f32 = dy_f32 != 0;
  a.w_f32 = w_f32 != 0;
  return norm_grad(a, workspace_bytes, stream);
}

moe_status moe_linear(const void* x, const void* w, const void* bias, int32_t bias_f32,
                      const void* residual, int32_t residual_f32, int32_t M, int32_t N, int32_t K,
                      int32_t act, void* pre, void* out, int32_t out_f32, moe_stream_t stream) {
  moe_status rc = check_linear(M, N, K, act);
  if (rc != MOE_OK || M == 0) return rc;
  MOE_REQ(x && w && out, MOE_ERR_INVALID_ARG, "x, w and out must be non-NULL");
  MOE_REQ(aligned(x, 16) && aligned(w, 16) && aligned(bias, 16) && aligned(residual, 16) && aligned(pre, 16) &&
              aligned(out, 16),
          MOE_ERR_INVALID_ARG, "misaligned pointer");
  MOE_REQ(residual != out || (residual_f32 != 0) == (out_f32 != 0), MOE_ERR_INVALID_ARG,
          "residual may be out only when both have one type");
  moe::LinearForm form;
  if ((rc = read_form(M == 1, &form)) != MOE_OK) return rc;
  int sms = 0, *status = nullptr;
  if ((rc = moe::api_device(&sms, &status)) != MOE_OK) return rc;
  moe::ProductArgs a{};
  a.a = w;
  a.b = x;
  a.P = N;
  a.Q = M;
  a.K = K;
  a.bias = bias;
  a.residual = residual;
  a.pre = pre;
  a.out = out;
  a.act = act;
  a.bias_f32 = bias_f32 != 0;
  a.res_f32 = residual_f32 != 0;
  a.out_f32 = out_f32 != 0;
  a.form = form;
  MOE_CUDA(moe::launch_product(a, sms, status, (cudaStream_t)stream), "linear launch");
  return MOE_OK;
}

size_t moe_linear_backward_workspace_size(int32_t M, int32_t N, int32_t K) {
  if (check_linear(M, N, K, MOE_ACT_NONE) != MOE_OK) return 0;
  return up256((size_t)M * N * 2) + (size_t)moe::kActGradRows * N * sizeof(float);
}

moe_status moe_linear_backward(const void* dout, int32_t dout_f32, const void* pre, const void* x,
                               const void* w, int32_t M, int32_t N, int32_t K, int32_t act, void* dx,
                               void* dw, int32_t dw_f32, float* db, void* workspace,
                               size_t workspace_bytes, moe_stream_t stream) {
  moe_status rc = check_linear(M, N, K, act);
  if (rc != MOE_OK) return rc;
  MOE_REQ(dx || dw || db, MOE_ERR_INVALID_ARG, "no output: give dx, dw or db");
  MOE_REQ(aligned(dx, 16) && aligned(dw, 16) && aligned(db, 4), MOE_ERR_INVALID_ARG, "misaligned pointer");
  if (M > 0) {
    MOE_REQ(dout && (x || !dw) && (w || !dx), MOE_ERR_INVALID_ARG,
            "dout, x (with dw) and w (with dx) must be non-NULL");
    MOE_REQ(pre || act == MOE_ACT_NONE, MOE_ERR_INVALID_ARG, "an activation needs pre");
    MOE_REQ(aligned(dout, 16) && aligned(pre, 16) && aligned(x, 16) && aligned(w, 16), MOE_ERR_INVALID_ARG,
            "misaligned pointer");
    const size_t need = moe_linear_backward_workspace_size(M, N, K);
    MOE_REQ(workspace_bytes >= need && workspace, MOE_ERR_WORKSPACE_TOO_SMALL,
            "linear backward workspace %zu < %zu bytes", workspace_bytes, need);
    MOE_REQ(aligned(workspace, 256), MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  }
  moe::LinearForm form = moe::kFormAuto;
  if (M > 0 && (rc = read_form(!dx && !dw, &form)) != MOE_OK) return rc;
  int sms = 0, *status = nullptr;
  if ((rc = moe::api_device(&sms, &status)) != MOE_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (M == 0) {
    if (dw) MOE_CUDA(cudaMemsetAsync(dw, 0, (size_t)N * K * (dw_f32 ? 4 : 2), st), "linear backward memset");
    if (db) MOE_CUDA(cudaMemsetAsync(db, 0, (size_t)N * 4, st), "linear backward memset");
    return MOE_OK;
  }
  const bool round = (act != MOE_ACT_NONE || dout_f32) && (dx || dw);
  const void* d = round ? workspace : dout;
  if (round || db) {
    moe::ActGradArgs g{};
    g.dout = dout;
    g.pre = pre;
    g.dpre = round ? workspace : nullptr;
    g.db = db;
    g.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256((size_t)M * N * 2));
    g.M = M;
    g.N = N;
    g.act = act;
    g.dout_f32 = dout_f32 != 0;
    MOE_CUDA(moe::launch_act_grad(g, sms, st), "linear backward launch (activation)");
  }
  if (dx) {
    moe::ProductArgs a{};
    a.a = w;
    a.a_mn = true;
    a.b = d;
    a.P = K;
    a.Q = M;
    a.K = N;
    a.out = dx;
    a.form = form;
    MOE_CUDA(moe::launch_product(a, sms, status, st), "linear backward launch (dx)");
  }
  if (dw) {
    moe::ProductArgs a{};
    a.a = x;
    a.a_mn = true;
    a.b = d;
    a.b_mn = true;
    a.P = K;
    a.Q = N;
    a.K = M;
    a.out = dw;
    a.out_f32 = dw_f32 != 0;
    a.form = form;
    MOE_CUDA(moe::launch_product(a, sms, status, st), "linear backward launch (dw)");
  }
  return MOE_OK;
}

}  // extern "C"
