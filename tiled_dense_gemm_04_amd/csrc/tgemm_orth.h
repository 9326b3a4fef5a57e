// tgemm_orth.h -- shared between the orthogonalisation's kernels (tgemm_orth.hip) and its host
// side (tgemm_orth_api.cpp).
#pragma once

#include "tgemm_internal.h"

namespace tgemm {

// One call: `batch` matrices G (R x C) to scale * NS(G). m = min(R, C), n = max(R, C), both
// padded to multiples of kOrthPad in the workspace (zeros there). The iterate keeps G's
// orientation: m x n, or n x m when G is tall.
constexpr int kOrthPad = 64;
constexpr int kOrthParts = 512;  // partial sums of squares per matrix, at most

struct OrthArgs {
  const void* G;
  _Float16* X;
  int64_t ldg, stride_g, ldx, stride_x;  // elements
  int batch, R, C, f32, tall;
  int mp, np;                            // padded m and n
  int nparts;                            // partial sums of squares per matrix
  float a, b, c, scale;
  // workspace (batch of each): sums of squares, the iterate's high and low halves twice, the
  // Gram matrix without its diagonal (high and low half) and its diagonal, the polynomial
  // likewise
  double* parts;
  _Float16 *hi[2], *lo[2], *E[2], *P[2];
  float *D, *DP;
};

hipError_t launch_orthogonalize(const OrthArgs& g, int steps, hipStream_t s, int device);

int current_device(int* device);  // tgemm_api.cpp

}  // namespace tgemm
