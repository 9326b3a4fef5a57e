// tgemm_expert.h -- shared between the kernels of the expert layer (tgemm_expert.hip: tokens sorted
// by expert and back; tgemm_expert_gemm.hip: the experts' products) and their host side
// (tgemm_expert_api.cpp).
#pragma once

#include "tgemm_internal.h"

namespace tgemm {

constexpr int kMaxExperts = 1024;

// f(row) for the rows first, first + n, ... before `rows` (64 bits: the row after the last may lie past 2^31).
template <typename F>
__host__ __device__ inline void every_nth_row(int64_t first, int64_t rows, int64_t n, F&& f) {
  for (int64_t r = first; r < rows; r += n) f(r);
}

// Sorting. Slot s = t * k + j holds the id of choice j of token t.
struct ExpertSortArgs {
  const void* ids;
  int64_t ldi;        // elements from one token's ids to the next's
  int tokens, k, n;   // n = tokens * k
  int experts, ids_i64;
  int *offsets, *order, *place;
  int* counts;        // workspace: kSortChunks x (experts + 1)
};
// Up to this many slots one launch sorts; beyond, two, over at most kSortChunks chunks of slots.
constexpr int kSortOneLaunch = 8192;
constexpr int kSortChunks = 256;
hipError_t launch_expert_sort(const ExpertSortArgs& g, hipStream_t s);

// Rows out to their places and back. Any index outside [0, rows) counts as no row.
struct ExpertRowsArgs {
  const _Float16 *src, *aux;  // gather: X; combine: Y; its gradient: dout and Y
  _Float16* dst;
  int64_t lds_, lda, ldd;     // strides of src, aux and dst, elements
  const int *place, *offsets; // offsets[experts]: the rows in use (null: rows behind them are left as they were)
  const void* weights;        // tokens x k, contiguous (null: ones)
  void* dweights;
  int tokens, k, rows, H, experts, w_f32;
};
hipError_t launch_expert_gather(const ExpertRowsArgs& g, hipStream_t s);
hipError_t launch_expert_combine(const ExpertRowsArgs& g, hipStream_t s);
hipError_t launch_expert_combine_grad(const ExpertRowsArgs& g, hipStream_t s);

// Products. Expert e owns rows offsets[e] .. offsets[e + 1] of A (and C, or B):
//   rows:    C[p, :] = ReLU?(A[p, :] op(B_e)),  B_e N x K (nt) or K x N;
//   weights: C_e (M x N) = A_e^T B_e over the expert's rows.
struct ExpertGemmArgs {
  const _Float16 *A, *B;
  _Float16* C;
  const int* offsets;
  int64_t lda, ldb, stride_b, ldc, stride_c;  // elements
  int rows, experts, M, N, K;                 // M: columns of A in the weights' form
  int relu, vec_c, zero_rest;
  int tiles_m, tiles_n;
  int mode;                                   // of the tile kernel, and the most tiles its rows' form goes over
  uint32_t max_tiles;
};
// k-tiles of BK of K values (an expert's rows in the weights' form: up to 2^31 - 1).
__host__ __device__ constexpr int k_tiles(int K, int BK) { return (int)(((uint32_t)K + (uint32_t)BK - 1) / (uint32_t)BK); }
enum ExpertForm { kExpertNT = 0, kExpertNN = 1, kExpertTN = 2 };
// Kernels of a product, by index (tooling ABI: the _cfg entry point). kExpertTiles mixes tiles of 256 x
// 256, 128 x 128 and, in the rows' form, 64 x 128; kExpert128 and kExpert256 are the same kernel held to one of them (but for
// edges).
enum ExpertConfig { kExpertGeneric = 0, kExpert32 = 1, kExpert128 = 2, kExpert256 = 3, kExpertTiles = 4, kExpert64 = 5, kExpertConfigs = 6 };
enum ExpertTileMode { kTilesAuto = 0, kTilesSmall = 1, kTilesBig = 2 };
constexpr int kExpertTileGroups = 256;  // workgroups of the tile kernel, each of which goes over tiles: one a compute unit
constexpr int expert_tile_m(int cfg) { return cfg == kExpert32 ? 32 : cfg == kExpert64 ? 64 : 128; }
// Workgroups of a launch. The rows' form of the others has one a tile: c rows of an expert need ceil(c
// / BM) tile rows, so all of them at most rows / BM + the number of experts that have one; and one
// tile row more where the rows behind the last group are to be zeroed by workgroups of no tile.
inline int64_t expert_gemm_groups(int cfg, int form, int64_t rows, int64_t experts, int64_t M, int64_t N) {
  const int64_t tn = ceil_div(N, 128);
  if (cfg == kExpert128 || cfg == kExpert256 || cfg == kExpertTiles) return kExpertTileGroups;
  if (form == kExpertTN) return experts * ceil_div(M, 128) * tn;
  return (rows / expert_tile_m(cfg) + (experts < rows ? experts : rows) + 1) * tn;
}
// The most tiles that the tile kernel has, whatever the division of the rows: of 128 x 128, and in the
// rows' form the halves of a last round.
inline int64_t expert_max_tiles(int form, int64_t rows, int64_t experts, int64_t M, int64_t N) {
  if (form == kExpertTN) return experts * (ceil_div(M, 128) + 1) * (ceil_div(N, 128) + 1);
  return (rows / 128 + 2 * (experts < rows ? experts : rows)) * (ceil_div(N, 128) + 1) + kExpertTileGroups;
}
hipError_t launch_expert_gemm(int cfg, ExpertForm form, const ExpertGemmArgs& g, hipStream_t s, int device);

int current_device(int* device);  // tgemm_api.cpp

}  // namespace tgemm
