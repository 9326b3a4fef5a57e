// tgemm_norm_api.cpp -- host side of the root-mean-square norm (declared in include/tgemm_ops.h):
// argument validation and launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tgemm_ops.h"
#include "tgemm_norm.h"

namespace {

static_assert(tgemm::kNormMaxK == TGEMM_NORM_MAX_K, "the header's limit");

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
// (The runtime takes fewer than 2^32 threads per launch.)
bool bad_dims(int64_t R, int64_t K) {
  if (R < 0 || K < 0 || R >= TGEMM_MAX_DIM || K > TGEMM_NORM_MAX_K) return true;
  return R * tgemm::norm_row_threads(K) > ((int64_t)1 << 32) - 2048;
}
bool bad_dtype(int dtype) { return dtype != TGEMM_DTYPE_F16 && dtype != TGEMM_DTYPE_F32; }
unsigned size_of(int dtype) { return dtype == TGEMM_DTYPE_F32 ? 4 : 2; }

}  // namespace

extern "C" {

int rmsnorm_f16(int64_t R, int64_t K, const void* X, int64_t ldx, const void* residual, int64_t ldr, int residual_dtype,
                const void* W, int w_dtype, float eps, void* residual_out, int64_t ldro, void* Y, int64_t ldy, void* Q,
                int64_t ldq, float* scale, void* stream) {
  if (bad_dims(R, K)) return TGEMM_EINVAL_DIM;
  const bool has_r = residual != nullptr;
  if (bad_dtype(w_dtype) || (has_r && bad_dtype(residual_dtype)) || !(eps >= 0.0f)) return TGEMM_EINVAL_DIM;
  const int64_t kmin = K > 1 ? K : 1;
  if (ldx < kmin || (has_r && ldr < kmin) || (residual_out != nullptr && ldro < kmin) || (Y != nullptr && ldy < kmin) ||
      (Q != nullptr && ldq < kmin))
    return TGEMM_EINVAL_LD;
  if (R == 0 || K == 0) return TGEMM_OK;
  if (X == nullptr || W == nullptr || (Y == nullptr && Q == nullptr) || (Q == nullptr) != (scale == nullptr) ||
      (residual_out != nullptr && !has_r))
    return TGEMM_ENULL;
  if (off(X, 2) || off(Y, 2) || off(W, size_of(w_dtype)) || off(scale, 4) ||
      (has_r && (off(residual, size_of(residual_dtype)) || off(residual_out, size_of(residual_dtype)))))
    return TGEMM_EALIGN;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  tgemm::NormArgs g;
  g.X = static_cast<const _Float16*>(X);
  g.Rin = residual;
  g.W = W;
  g.Rout = residual_out;
  g.Y = static_cast<_Float16*>(Y);
  g.Q = static_cast<uint8_t*>(Q);
  g.S = scale;
  g.ldx = ldx;
  g.ldr = ldr;
  g.ldro = ldro;
  g.ldy = ldy;
  g.ldq = ldq;
  g.R = (int)R;
  g.K = (int)K;
  g.KB = (int)tgemm::ceil_div(K, tgemm::kFp8Block);
  g.w_f32 = w_dtype == TGEMM_DTYPE_F32;
  g.eps = eps;
  const int res = !has_r ? tgemm::kResNone : residual_dtype == TGEMM_DTYPE_F32 ? tgemm::kResF32 : tgemm::kResF16;
  return tgemm::launch_rmsnorm(g, res, static_cast<hipStream_t>(stream)) == hipSuccess ? TGEMM_OK : TGEMM_ELAUNCH;
}

int64_t rmsnorm_f16_backward_workspace_bytes(int64_t R, int64_t K) {
  if (bad_dims(R, K)) return TGEMM_EINVAL_DIM;
  return R == 0 || K == 0 ? 0 : (int64_t)tgemm::norm_grad_groups(R, K) * K * 4;
}

int rmsnorm_f16_backward(int64_t R, int64_t K, const void* dY, int64_t lddy, const void* H, int64_t ldh, int h_dtype,
                         const void* W, int w_dtype, float eps, const void* dH, int64_t lddh, void* dX,
                         int64_t lddx, void* dR, int64_t lddr, void* dW, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  if (bad_dims(R, K) || bad_dtype(h_dtype) || bad_dtype(w_dtype) || !(eps >= 0.0f)) return TGEMM_EINVAL_DIM;
  const int64_t kmin = K > 1 ? K : 1;
  if (lddy < kmin || ldh < kmin || lddx < kmin || (dH != nullptr && lddh < kmin) || (dR != nullptr && lddr < kmin))
    return TGEMM_EINVAL_LD;
  if (K == 0 || (R == 0 && dW == nullptr)) return TGEMM_OK;
  if (R > 0 && (dY == nullptr || H == nullptr || dX == nullptr)) return TGEMM_ENULL;
  if (W == nullptr || (R > 0 && dW != nullptr && workspace == nullptr)) return TGEMM_ENULL;
  const unsigned hs = size_of(h_dtype), ws = size_of(w_dtype);
  if (off(dY, 2) || off(dX, 2) || off(H, hs) || off(dH, hs) || off(dR, hs) || off(W, ws) || off(dW, ws) ||
      off(workspace, 256))
    return TGEMM_EALIGN;
  if (dW != nullptr && workspace_bytes < rmsnorm_f16_backward_workspace_bytes(R, K)) return TGEMM_EWORKSPACE;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  tgemm::NormGradArgs g;
  g.dY = static_cast<const _Float16*>(dY);
  g.H = H;
  g.W = W;
  g.dH = dH;
  g.dX = static_cast<_Float16*>(dX);
  g.dR = dR;
  g.dW = dW;
  g.parts = static_cast<float*>(workspace);
  g.lddy = lddy;
  g.ldh = ldh;
  g.lddh = lddh;
  g.lddx = lddx;
  g.lddr = lddr;
  g.R = (int)R;
  g.K = (int)K;
  g.w_f32 = w_dtype == TGEMM_DTYPE_F32;
  g.eps = eps;
  g.groups = R == 0 ? 0 : tgemm::norm_grad_groups(R, K);
  return tgemm::launch_rmsnorm_backward(g, h_dtype == TGEMM_DTYPE_F32, static_cast<hipStream_t>(stream)) == hipSuccess
             ? TGEMM_OK
             : TGEMM_ELAUNCH;
}

}  // extern "C"
