// tgemm_norm.h -- shared between the root-mean-square norm's kernels (tgemm_norm.hip) and its host
// side (tgemm_norm_api.cpp).
#pragma once

#include "tgemm_internal.h"

namespace tgemm {

constexpr int kNormMaxK = 16384;     // a row is held in one workgroup's registers
// Threads that hold a row of K values.
constexpr int norm_row_threads(int64_t K) {
  return K <= 128 ? 16 : K <= 256 ? 32 : K <= 1024 ? 64 : K <= 4096 ? 256 : K <= 8192 ? 512 : 1024;
}

// Residual types (kNone: no residual, the norm is of X itself).
enum NormResidual { kResNone = 0, kResF16 = 1, kResF32 = 2 };

struct NormArgs {
  const _Float16* X;
  const void *Rin, *W;
  void* Rout;
  _Float16* Y;     // any of Rout, Y, and Q and S together may be null
  uint8_t* Q;
  float* S;
  int64_t ldx, ldr, ldro, ldy, ldq;  // elements
  int R, K, KB, w_f32;
  float eps;
};
hipError_t launch_rmsnorm(const NormArgs& g, int residual, hipStream_t s);

struct NormGradArgs {
  const _Float16* dY;
  const void *H, *W, *dH;  // dH may be null; H and dH have the residual's type
  _Float16* dX;
  void *dR, *dW;           // dR (the residual's type) and dW (W's type) may be null
  float* parts;            // groups x K partial sums of dW
  int64_t lddy, ldh, lddh, lddx, lddr;
  int R, K, w_f32, groups;
  float eps;
};
// Workgroups of the backward kernel (each leaves one row of partial sums).
int norm_grad_groups(int64_t R, int64_t K);
hipError_t launch_rmsnorm_backward(const NormGradArgs& g, bool h_f32, hipStream_t s);

int current_device(int* device);  // tgemm_api.cpp

}  // namespace tgemm
