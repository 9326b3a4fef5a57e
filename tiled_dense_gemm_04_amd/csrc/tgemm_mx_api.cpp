// tgemm_mx_api.cpp -- host side of the MXFP4 entry points (declared in include/tgemm_ops.h):
// argument validation, kernel choice and launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tgemm_ops.h"
#include "tgemm_mx.h"

namespace {

using tgemm::MxGemmArgs;

// The kernels index rows and columns of a tile past the matrix's edge in 32 bits.
constexpr int64_t kMaxDim = TGEMM_MX_MAX_DIM;
// The runtime takes fewer than 2^32 threads per launch; the widest kernels here have 512 a
// workgroup (the skinny one up to 1024).
constexpr int64_t kMaxGrid = ((int64_t)1 << 23) - 1, kMaxSkinnyN = 16 * (((int64_t)1 << 22) - 1);
// Blocks along the rows of a matrix that is quantised or decoded: 128 per workgroup of 256 threads.
constexpr int64_t kMaxBlocks = ((int64_t)1 << 31) - 128;

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
bool aligned16(const void* p) { return (addr(p) & 15u) == 0; }
int64_t blocks(int64_t k) { return tgemm::ceil_div(k, tgemm::kMxBlock); }
bool bad_dim(int64_t d) { return d < 0 || d > kMaxDim; }
// An MXFP4 matrix's row strides hold its whole blocks.
bool bad_ld(int64_t k, int64_t ldq, int64_t lds) {
  const int64_t kb = blocks(k) > 0 ? blocks(k) : 1;
  return ldq < kb * tgemm::kMxBlockBytes || lds < kb;
}

int validate(bool f16_a, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA, int64_t ldsa,
             const void* B, int64_t ldb, const void* SB, int64_t ldsb, const void* C, int64_t ldc) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return TGEMM_EINVAL_DIM;
  if (f16_a ? lda < (K > 1 ? K : 1) : bad_ld(K, lda, ldsa)) return TGEMM_EINVAL_LD;
  if (bad_ld(K, ldb, ldsb) || ldc < (N > 1 ? N : 1)) return TGEMM_EINVAL_LD;
  if (M == 0 || N == 0) return TGEMM_OK;
  if (C == nullptr) return TGEMM_ENULL;
  if (K > 0 && (A == nullptr || B == nullptr || SB == nullptr || (!f16_a && SA == nullptr))) return TGEMM_ENULL;
  if ((addr(C) & 1u) || (f16_a && (addr(A) & 1u))) return TGEMM_EALIGN;
  return TGEMM_OK;
}

// The fast kernels copy 16-byte chunks (a whole MX block, 16 scales, 8 binary16 values) and
// address a 256-row operand tile through a 32-bit buffer range. The skinny kernel takes scales
// and binary16 A of any alignment.
bool rows_eligible(const void* p, int64_t ld) { return aligned16(p) && ld % 16 == 0 && ld <= 2 * TGEMM_FAST_MAX_LD; }
bool f16_eligible(int64_t K, const void* A, int64_t lda) {
  return aligned16(A) && lda % 8 == 0 && K % 8 == 0 && lda <= TGEMM_FAST_MAX_LD;
}
bool tiles_eligible(bool f16_a, int64_t K, const void* A, int64_t lda, const void* SA, int64_t ldsa, const void* SB,
                    int64_t ldsb) {
  return rows_eligible(SB, ldsb) && (f16_a ? f16_eligible(K, A, lda) : rows_eligible(SA, ldsa));
}

// Kernel choice of a fast-eligible call, by rounds of workgroups over the 256 compute units. One
// round at K = 4096 measured (microseconds beyond the launch; all scale with K):
//   A in MXFP4:    skinny 4 (up to 16 rows), 5 (48), 8 (64); 64 x 128 tiles 11 to 13; 128 x 128
//                  14 to 15; 256 x 256 28 to 36;
//   A in binary16: skinny 5, 9, 12; 128 x 128 tiles 42; 256 x 256 84 to 100.
// The skinny kernel takes 64 rows of A by 16 of the weight per workgroup. (128 x 128 is the smallest
// tile with binary16 A: at N = 4096 a round of it serves 129 rows or 1024 in the same 42 us.)
int64_t skinny_groups(int64_t M, int64_t N) { return tgemm::ceil_div(M, tgemm::kMxSkinnyTile) * tgemm::ceil_div(N, 16); }
int choose(bool f16_a, int64_t M, int64_t N) {
  const int64_t skinny = skinny_groups(M, N);
  const int64_t t128 = tgemm::ceil_div(M, 128) * tgemm::ceil_div(N, 128);
  const int64_t t64 = tgemm::ceil_div(M, 64) * tgemm::ceil_div(N, 128);
  const bool narrow = N <= kMaxSkinnyN;
  if (M <= 32 && narrow) return tgemm::kMxSkinny;
  if (f16_a) {
    // up to three rounds of the skinny kernel cost less than one of 128 x 128 tiles, and two
    // rounds of those about one of 256 x 256 (512 tiles: 80 against 85 us; 576: 88 against 67)
    if (M <= tgemm::kMxSkinnyRows && skinny <= 3 * 256) return tgemm::kMxSkinny;
    return t128 <= 512 ? tgemm::kMx128 : tgemm::kMx256;
  }
  if (M <= tgemm::kMxSkinnyTile && skinny <= 256) return tgemm::kMxSkinny;
  if (t64 <= 256) return tgemm::kMx64;
  return t128 <= 256 ? tgemm::kMx128 : tgemm::kMx256;
}

// Binary16 A or scales that the tiles cannot take (their alignment or stride, K): the skinny kernel
// up to a number of rounds of its workgroups, then the generic one.
//   A in binary16, 4 rounds: K = 4095: 61 us (65 x 8192), 74 (100 x 8192), 90 (128 x 8192), 88 (256 x
//   4096), the generic kernel 101 to 117; K = 1001: 32 to 42 against 30 to 33. 8 rounds: 152 (200 x
//   8192 x 4095) against 120, 72 (200 x 8192 x 1001) against 32.
//   A in MXFP4, 16 rounds: 109 us (256 x 16384 x 4095), 39 (x 1001), the generic kernel 151 and 42.
//   32 rounds: 213 (256 x 32768 x 4095) against 181, 79 against 55.
int choose_any(bool f16_a, int64_t M, int64_t N) {
  return M <= tgemm::kMxSkinnyRows && N <= kMaxSkinnyN && skinny_groups(M, N) <= (f16_a ? 4 : 16) * 256 ? tgemm::kMxSkinny
                                                                                                   : tgemm::kMxGeneric;
}

constexpr int kSelectNoop = -100, kSelectZeroFill = -101;

int select(bool f16_a, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA, int64_t ldsa,
           const void* B, int64_t ldb, const void* SB, int64_t ldsb, const void* C, int64_t ldc) {
  const int v = validate(f16_a, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc);
  if (v != TGEMM_OK) return v;
  if (M == 0 || N == 0) return kSelectNoop;
  if (K == 0) return kSelectZeroFill;
  if (!rows_eligible(B, ldb) || (!f16_a && !rows_eligible(A, lda))) return tgemm::kMxGeneric;
  const int cfg = choose(f16_a, M, N);
  if (cfg == tgemm::kMxSkinny) return cfg;
  return tiles_eligible(f16_a, K, A, lda, SA, ldsa, SB, ldsb) ? cfg : choose_any(f16_a, M, N);
}

// Runs the product; force: a kernel index, or -1 for the choice.
int run(bool f16_a, int force, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA,
        int64_t ldsa, const void* B, int64_t ldb, const void* SB, int64_t ldsb, void* C, int64_t ldc, int relu,
        void* stream) {
  int cfg = select(f16_a, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc);
  if (cfg == kSelectNoop) return TGEMM_OK;
  if (cfg < 0 && cfg != kSelectZeroFill) return cfg;
  if (force >= 0 && cfg != kSelectZeroFill) {
    if (force != tgemm::kMxGeneric) {
      if (!rows_eligible(B, ldb) || (!f16_a && !rows_eligible(A, lda))) return TGEMM_EINVAL_CFG;
      if (force == tgemm::kMxSkinny ? M > tgemm::kMxSkinnyRows || N > kMaxSkinnyN
                                    : !tiles_eligible(f16_a, K, A, lda, SA, ldsa, SB, ldsb))
        return TGEMM_EINVAL_CFG;
      if (force == tgemm::kMx64 && f16_a) return TGEMM_EINVAL_CFG;
    }
    cfg = force;
  }
  if (cfg != tgemm::kMxSkinny && cfg != kSelectZeroFill &&
      tgemm::ceil_div(M, tgemm::mx_tile_m(cfg)) * tgemm::ceil_div(N, tgemm::mx_tile_n(cfg)) > kMaxGrid)
    return TGEMM_EINVAL_DIM;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (cfg == kSelectZeroFill) {
    e = tgemm::launch_zero_fill(static_cast<_Float16*>(C), (int)M, (int)N, ldc, s);
  } else {
    MxGemmArgs g;
    g.A = A;
    g.SA = static_cast<const uint8_t*>(SA);
    g.B = static_cast<const uint8_t*>(B);
    g.SB = static_cast<const uint8_t*>(SB);
    g.C = static_cast<_Float16*>(C);
    g.lda = lda;
    g.ldsa = ldsa;
    g.ldb = ldb;
    g.ldsb = ldsb;
    g.ldc = ldc;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.KB = (int)blocks(K);
    g.relu = relu != 0;
    g.vec_c = aligned16(C) && ldc % 8 == 0;
    g.tiles_m = g.tiles_n = 0;
    e = tgemm::launch_mxfp4(cfg, f16_a, g, s, dev);
  }
  return e == hipSuccess ? TGEMM_OK : TGEMM_ELAUNCH;
}

}  // namespace

extern "C" {

int mxfp4_quant(int64_t R, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, void* scale, int64_t lds,
                void* QT, int64_t ldqt, void* scale_t, int64_t ldst, void* stream) {
  if (bad_dim(R) || bad_dim(K)) return TGEMM_EINVAL_DIM;
  const bool rows = Q != nullptr || scale != nullptr, cols = QT != nullptr || scale_t != nullptr;
  if (ldx < (K > 1 ? K : 1) || (rows && bad_ld(K, ldq, lds)) || (cols && bad_ld(R, ldqt, ldst))) return TGEMM_EINVAL_LD;
  if (R == 0 || K == 0) return TGEMM_OK;
  if (X == nullptr || (!rows && !cols)) return TGEMM_ENULL;
  if ((rows && (Q == nullptr || scale == nullptr)) || (cols && (QT == nullptr || scale_t == nullptr))) return TGEMM_ENULL;
  if (addr(X) & 1u) return TGEMM_EALIGN;
  if (R * blocks(K) > kMaxBlocks) return TGEMM_EINVAL_DIM;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  tgemm::MxQuantArgs q;
  q.X = static_cast<const _Float16*>(X);
  q.Q = static_cast<uint8_t*>(Q);
  q.S = static_cast<uint8_t*>(scale);
  q.QT = static_cast<uint8_t*>(QT);
  q.ST = static_cast<uint8_t*>(scale_t);
  q.ldx = ldx;
  q.ldq = ldq;
  q.lds = lds;
  q.ldqt = ldqt;
  q.ldst = ldst;
  q.R = (int)R;
  q.K = (int)K;
  return tgemm::launch_quant_mxfp4(q, static_cast<hipStream_t>(stream)) == hipSuccess ? TGEMM_OK : TGEMM_ELAUNCH;
}

int mxfp4_dequant(int64_t R, int64_t K, const void* Q, int64_t ldq, const void* scale, int64_t lds, void* X,
                  int64_t ldx, void* stream) {
  if (bad_dim(R) || bad_dim(K)) return TGEMM_EINVAL_DIM;
  if (ldx < (K > 1 ? K : 1) || bad_ld(K, ldq, lds)) return TGEMM_EINVAL_LD;
  if (R == 0 || K == 0) return TGEMM_OK;
  if (X == nullptr || Q == nullptr || scale == nullptr) return TGEMM_ENULL;
  if (addr(X) & 1u) return TGEMM_EALIGN;
  if (R * blocks(K) > kMaxBlocks) return TGEMM_EINVAL_DIM;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  tgemm::MxDequantArgs q;
  q.Q = static_cast<const uint8_t*>(Q);
  q.S = static_cast<const uint8_t*>(scale);
  q.X = static_cast<_Float16*>(X);
  q.ldq = ldq;
  q.lds = lds;
  q.ldx = ldx;
  q.R = (int)R;
  q.K = (int)K;
  return tgemm::launch_dequant_mxfp4(q, static_cast<hipStream_t>(stream)) == hipSuccess ? TGEMM_OK : TGEMM_ELAUNCH;
}

int mxfp4_gemm(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* scale_a, int64_t ldsa,
               const void* B, int64_t ldb, const void* scale_b, int64_t ldsb, void* C, int64_t ldc, int relu,
               void* stream) {
  return run(false, -1, M, N, K, A, lda, scale_a, ldsa, B, ldb, scale_b, ldsb, C, ldc, relu, stream);
}

int mxfp4_gemm_f16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                   const void* scale_b, int64_t ldsb, void* C, int64_t ldc, int relu, void* stream) {
  return run(true, -1, M, N, K, A, lda, nullptr, 0, B, ldb, scale_b, ldsb, C, ldc, relu, stream);
}

int mxfp4_gemm_cfg(int idx, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* scale_a,
                   int64_t ldsa, const void* B, int64_t ldb, const void* scale_b, int64_t ldsb, void* C, int64_t ldc,
                   int relu, void* stream) {
  if (idx < 0 || idx >= tgemm::kMxConfigs) return TGEMM_EINVAL_CFG;
  return run(false, idx, M, N, K, A, lda, scale_a, ldsa, B, ldb, scale_b, ldsb, C, ldc, relu, stream);
}

int mxfp4_gemm_f16_cfg(int idx, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                       int64_t ldb, const void* scale_b, int64_t ldsb, void* C, int64_t ldc, int relu, void* stream) {
  if (idx < 0 || idx >= tgemm::kMxConfigs) return TGEMM_EINVAL_CFG;
  return run(true, idx, M, N, K, A, lda, nullptr, 0, B, ldb, scale_b, ldsb, C, ldc, relu, stream);
}

int mxfp4_select_config(int f16_a, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* scale_a, int64_t ldsa, const void* B, int64_t ldb, const void* scale_b,
                              int64_t ldsb, const void* C, int64_t ldc) {
  return select(f16_a != 0, M, N, K, A, lda, scale_a, ldsa, B, ldb, scale_b, ldsb, C, ldc);
}

}  // extern "C"
