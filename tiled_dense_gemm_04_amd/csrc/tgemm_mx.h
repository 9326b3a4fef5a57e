// tgemm_mx.h -- shared between the MXFP4 kernels (tgemm_mx.hip) and their host side
// (tgemm_mx_api.cpp).
#pragma once

#include "tgemm_internal.h"

namespace tgemm {

// One MX block: 32 E2M1 codes (16 bytes, the even k in the low half of a byte) sharing one
// E8M0 scale byte s that stands for 2^(s - 127) (255: NaN).
constexpr int kMxBlock = 32, kMxBlockBytes = 16;

// Quantiser: X (R x K binary16) to codes and scales along its rows (Q, S) and / or its columns
// (QT, ST: X^T quantised along R). A pair of null pointers is not written.
struct MxQuantArgs {
  const _Float16* X;
  uint8_t *Q, *S, *QT, *ST;
  int64_t ldx, ldq, lds, ldqt, ldst;  // elements (X), bytes (the others)
  int R, K;
};
hipError_t launch_quant_mxfp4(const MxQuantArgs& q, hipStream_t s);

struct MxDequantArgs {
  const uint8_t *Q, *S;
  _Float16* X;
  int64_t ldq, lds, ldx;
  int R, K;
};
hipError_t launch_dequant_mxfp4(const MxDequantArgs& q, hipStream_t s);

// C (M x N binary16) = ReLU?(A B^T): A is M x K, MXFP4 codes with scales SA (mxfp4_gemm) or
// binary16 (mxfp4_gemm_f16, SA null), B is N x K MXFP4 codes with scales SB.
struct MxGemmArgs {
  const void* A;
  const uint8_t *SA, *B, *SB;
  _Float16* C;
  int64_t lda, ldsa, ldb, ldsb, ldc;  // lda: bytes of codes, or binary16 elements
  int M, N, K, KB;                    // KB = ceil(K / 32)
  int relu, vec_c;                    // vec_c: C 16-byte aligned and ldc a multiple of 8
  int tiles_m, tiles_n;
};

// The kernels of a product, by index (tooling ABI: the _cfg entry points).
enum MxConfig { kMxGeneric = 0, kMxSkinny = 1, kMx128 = 2, kMx256 = 3, kMx64 = 4, kMxConfigs = 5 };
constexpr int mx_tile_m(int cfg) { return cfg == kMx256 ? 256 : cfg == kMx64 ? 64 : 128; }
constexpr int mx_tile_n(int cfg) { return cfg == kMx256 ? 256 : 128; }
constexpr int kMxSkinnyTile = 64;   // rows of A per workgroup of the skinny kernel
constexpr int kMxSkinnyRows = 256;  // its largest M
hipError_t launch_mxfp4(int cfg, bool f16_a, const MxGemmArgs& g, hipStream_t s, int device);

// The current device, if it is one the library runs on (tgemm_api.cpp).
int current_device(int* device);

}  // namespace tgemm
