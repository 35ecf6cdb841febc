// extern "C" entry points of the operators around the experts' products:
// argument checks and launches.
#include <stdarg.h>
#include <stdio.h>

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
  MOE_CUDA(moe::launch_unpermute_grad(a, status, (cudaStream_t)stream), "unpermute backward launch");
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
  MOE_CUDA(moe::launch_layernorm(a, (cudaStream_t)stream), "layernorm launch");
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

}  // extern "C"
