// tgemm_expert_api.cpp -- host side of the expert layer's entry points (declared in
// include/tgemm_ops.h): argument validation, kernel choice and launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tgemm_ops.h"
#include "tgemm_expert.h"

namespace {

using tgemm::ExpertGemmArgs;
using tgemm::ExpertRowsArgs;

static_assert(tgemm::kMaxExperts == TGEMM_MAX_EXPERTS, "the header's limit");

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
bool bad_dim(int64_t d) { return d < 0 || d >= TGEMM_MAX_DIM; }
bool bad_dtype(int dtype) { return dtype != TGEMM_DTYPE_F16 && dtype != TGEMM_DTYPE_F32; }
bool bad_experts(int64_t e) { return e < 1 || e > TGEMM_MAX_EXPERTS; }
int64_t at_least_1(int64_t v) { return v > 1 ? v : 1; }
const int* ints(const void* p) { return static_cast<const int*>(p); }
const _Float16* halves(const void* p) { return static_cast<const _Float16*>(p); }

// Tokens and their slots: a slot's index, and the threads of a launch with a wave per slot, stay
// below 2^32.
int check_slots(int64_t tokens, int64_t k) {
  if (bad_dim(tokens) || bad_dim(k)) return TGEMM_EINVAL_DIM;
  return tokens * k > TGEMM_MAX_SLOTS ? TGEMM_EINVAL_DIM : TGEMM_OK;
}
// Rows of H values of `tokens` tokens: eight values a thread, and as many threads below 2^32.
int check_rows(int64_t tokens, int64_t k, int64_t rows, int64_t H) {
  const int v = check_slots(tokens, k);
  if (v != TGEMM_OK) return v;
  if (bad_dim(rows) || bad_dim(H)) return TGEMM_EINVAL_DIM;
  return tokens * tgemm::ceil_div(H, 8) > ((int64_t)1 << 32) - (1 << 16) ? TGEMM_EINVAL_DIM : TGEMM_OK;
}

int finish(hipError_t e) { return e == hipSuccess ? TGEMM_OK : TGEMM_ELAUNCH; }

int64_t sort_workspace(int64_t n, int64_t experts) {
  return n <= tgemm::kSortOneLaunch ? 0 : (int64_t)tgemm::kSortChunks * (experts + 1) * 4;
}

// The tile kernels copy 16-byte chunks along each operand's contiguous dimension and address a
// 256-row tile through a 32-bit buffer range.
bool chunks(const void* p, int64_t ld, int64_t width) {
  return !off(p, 16) && ld % 8 == 0 && width % 8 == 0 && ld <= TGEMM_FAST_MAX_LD;
}

// Kernel of a product whose operands the tiles take, by the rows an expert has on average (uneven
// experts; microseconds of the tiles of 32 rows, of 64, and of 128 and 256):
//   32 rows: 112, 120, 137 (64 experts, 2048 x 2048), 15.6, 20.1, 16.0 (8);
//   64: 142, 128, 136 (64), 42, 39, 51 (16), 20.6, 19.3, 17.3 (8), 14.1, 18.5, 13.9 (1);
//   96: 174, 141, 144 (64), 51, 40, 48 (16), 20.1, 20.3, 19.7 (8);   128: 212, -, 152 (64), 61, 50, 52 (16).
// So 64 rows where the small tiles would be more than one round of halves.
int choose(int form, int64_t rows, int64_t experts, int64_t N) {
  const int64_t met = rows < experts ? at_least_1(rows) : experts, each = rows / met;
  if (form == tgemm::kExpertTN) return tgemm::kExpertTiles;
  if (each <= 48) return tgemm::kExpert32;
  const bool one_round = met * tgemm::ceil_div(N, 128) <= tgemm::kExpertTileGroups / 2;
  return each <= 96 && !one_round ? tgemm::kExpert64 : tgemm::kExpertTiles;
}

int validate(int form, int64_t rows, int64_t experts, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
             const void* offsets, const void* B, int64_t ldb, int64_t stride_b, const void* C, int64_t ldc,
             int64_t stride_c) {
  const bool tn = form == tgemm::kExpertTN;
  if (bad_experts(experts) || bad_dim(rows) || bad_dim(M) || bad_dim(N) || bad_dim(K)) return TGEMM_EINVAL_DIM;
  if (lda < at_least_1(tn ? M : K) || ldb < at_least_1(form == tgemm::kExpertNT ? K : N) || ldc < at_least_1(N) ||
      stride_b < 0)
    return TGEMM_EINVAL_LD;
  // results of the experts may not overlap
  if (tn && experts > 1 && M > 0 && stride_c < (M - 1) * ldc + N) return TGEMM_EINVAL_LD;
  if (N == 0 || (tn ? M == 0 : rows == 0)) return TGEMM_OK;
  const bool reads = tn ? rows > 0 : K > 0;
  if (C == nullptr || offsets == nullptr || (reads && (A == nullptr || B == nullptr))) return TGEMM_ENULL;
  return off(A, 2) || off(B, 2) || off(C, 2) || off(offsets, 4) ? TGEMM_EALIGN : TGEMM_OK;
}

constexpr int kSelectNoop = -100;

// (K == 0 takes the generic kernel, which then reads neither operand.)
bool tiles_eligible(int form, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                    int64_t stride_b) {
  if (form == tgemm::kExpertTN) return chunks(A, lda, M) && chunks(B, ldb, N);
  return K > 0 && stride_b % 8 == 0 && chunks(A, lda, K) && chunks(B, ldb, form == tgemm::kExpertNT ? K : N);
}

int select(int form, int64_t rows, int64_t experts, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
           const void* offsets, const void* B, int64_t ldb, int64_t stride_b, const void* C, int64_t ldc,
           int64_t stride_c) {
  const int v = validate(form, rows, experts, M, N, K, A, lda, offsets, B, ldb, stride_b, C, ldc, stride_c);
  if (v != TGEMM_OK) return v;
  if (N == 0 || (form == tgemm::kExpertTN ? M == 0 : rows == 0)) return kSelectNoop;
  return tiles_eligible(form, M, N, K, A, lda, B, ldb, stride_b) ? choose(form, rows, experts, N) : tgemm::kExpertGeneric;
}

int run(int force, int form, int64_t rows, int64_t experts, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
        const void* offsets, const void* B, int64_t ldb, int64_t stride_b, void* C, int64_t ldc, int64_t stride_c,
        int relu, int zero_rest, void* stream) {
  int cfg = select(form, rows, experts, M, N, K, A, lda, offsets, B, ldb, stride_b, C, ldc, stride_c);
  if (cfg == kSelectNoop) return TGEMM_OK;
  if (cfg < 0) return cfg;
  if (force >= 0) {
    if (force != tgemm::kExpertGeneric && !tiles_eligible(form, M, N, K, A, lda, B, ldb, stride_b)) return TGEMM_EINVAL_CFG;
    if ((force == tgemm::kExpert32 || force == tgemm::kExpert64) && form == tgemm::kExpertTN) return TGEMM_EINVAL_CFG;
    cfg = force;
  }
  // the runtime takes fewer than 2^32 threads per launch, 512 a workgroup at most; the tile kernel counts
  // its tiles in 32 bits
  if (tgemm::expert_gemm_groups(cfg, form, rows, experts, M, N) >= ((int64_t)1 << 23) ||
      tgemm::expert_max_tiles(form, rows, experts, M, N) >= ((int64_t)1 << 31))
    return TGEMM_EINVAL_DIM;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  ExpertGemmArgs g;
  g.A = halves(A);
  g.B = halves(B);
  g.C = static_cast<_Float16*>(C);
  g.offsets = ints(offsets);
  g.lda = lda;
  g.ldb = ldb;
  g.stride_b = stride_b;
  g.ldc = ldc;
  g.stride_c = stride_c;
  g.rows = (int)rows;
  g.experts = (int)experts;
  g.M = (int)M;
  g.N = (int)N;
  g.K = (int)K;
  g.relu = relu != 0;
  g.vec_c = !off(C, 16) && ldc % 8 == 0 && stride_c % 8 == 0;
  g.zero_rest = zero_rest != 0;
  g.tiles_m = g.tiles_n = 0;
  return finish(tgemm::launch_expert_gemm(cfg, static_cast<tgemm::ExpertForm>(form), g, static_cast<hipStream_t>(stream), dev));
}

ExpertRowsArgs rows_args(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* place) {
  ExpertRowsArgs g{};
  g.place = ints(place);
  g.tokens = (int)tokens;
  g.k = (int)k;
  g.rows = (int)rows;
  g.H = (int)H;
  return g;
}

}  // namespace

extern "C" {

int64_t expert_sort_workspace_bytes(int64_t tokens, int64_t k, int64_t experts) {
  const int v = check_slots(tokens, k);
  if (v != TGEMM_OK) return v;
  return bad_experts(experts) ? TGEMM_EINVAL_DIM : sort_workspace(tokens * k, experts);
}

int expert_sort(int64_t tokens, int64_t k, int64_t experts, const void* ids, int64_t ldi, int ids_type, void* offsets,
                void* order, void* place, void* workspace, int64_t workspace_bytes, void* stream) {
  const int v = check_slots(tokens, k);
  if (v != TGEMM_OK) return v;
  if (bad_experts(experts) || (ids_type != TGEMM_INDEX_I32 && ids_type != TGEMM_INDEX_I64)) return TGEMM_EINVAL_DIM;
  if (ldi < at_least_1(k)) return TGEMM_EINVAL_LD;
  const int64_t n = tokens * k, need = sort_workspace(n, experts);
  if (offsets == nullptr || (n > 0 && (ids == nullptr || order == nullptr || place == nullptr)) ||
      (need > 0 && workspace == nullptr))
    return TGEMM_ENULL;
  if (off(offsets, 4) || off(order, 4) || off(place, 4) || off(ids, ids_type == TGEMM_INDEX_I64 ? 8 : 4) ||
      off(workspace, 256))
    return TGEMM_EALIGN;
  if (workspace_bytes < need) return TGEMM_EWORKSPACE;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  tgemm::ExpertSortArgs g;
  g.ids = ids;
  g.ldi = ldi;
  g.tokens = (int)tokens;
  g.k = (int)k;
  g.n = (int)n;
  g.experts = (int)experts;
  g.ids_i64 = ids_type == TGEMM_INDEX_I64;
  g.offsets = static_cast<int*>(offsets);
  g.order = static_cast<int*>(order);
  g.place = static_cast<int*>(place);
  g.counts = static_cast<int*>(workspace);
  return finish(tgemm::launch_expert_sort(g, static_cast<hipStream_t>(stream)));
}

int expert_gather_f16(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* X, int64_t ldx, const void* place,
                      void* XS, int64_t ldxs, const void* offsets, int64_t experts, void* stream) {
  const int v = check_rows(tokens, k, rows, H);
  if (v != TGEMM_OK) return v;
  if (offsets != nullptr && bad_experts(experts)) return TGEMM_EINVAL_DIM;
  if (ldx < at_least_1(H) || ldxs < at_least_1(H)) return TGEMM_EINVAL_LD;
  if (rows == 0 || H == 0 || (offsets == nullptr && tokens * k == 0)) return TGEMM_OK;
  if (XS == nullptr || (tokens * k > 0 && (X == nullptr || place == nullptr))) return TGEMM_ENULL;
  if (off(X, 2) || off(XS, 2) || off(place, 4) || off(offsets, 4)) return TGEMM_EALIGN;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  ExpertRowsArgs g = rows_args(tokens, k, rows, H, place);
  g.src = halves(X);
  g.lds_ = ldx;
  g.dst = static_cast<_Float16*>(XS);
  g.ldd = ldxs;
  g.offsets = ints(offsets);
  g.experts = (int)experts;
  return finish(tgemm::launch_expert_gather(g, static_cast<hipStream_t>(stream)));
}

int expert_combine_f16(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* Y, int64_t ldy, const void* place,
                       const void* weights, int w_dtype, void* OUT, int64_t ldo, void* stream) {
  const int v = check_rows(tokens, k, rows, H);
  if (v != TGEMM_OK) return v;
  if (weights != nullptr && bad_dtype(w_dtype)) return TGEMM_EINVAL_DIM;
  if (ldy < at_least_1(H) || ldo < at_least_1(H)) return TGEMM_EINVAL_LD;
  if (tokens == 0 || H == 0) return TGEMM_OK;
  if (OUT == nullptr || (k > 0 && (place == nullptr || (rows > 0 && Y == nullptr)))) return TGEMM_ENULL;
  if (off(Y, 2) || off(OUT, 2) || off(place, 4) || off(weights, w_dtype == TGEMM_DTYPE_F32 ? 4 : 2)) return TGEMM_EALIGN;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  ExpertRowsArgs g = rows_args(tokens, k, rows, H, place);
  g.src = halves(Y);
  g.lds_ = ldy;
  g.dst = static_cast<_Float16*>(OUT);
  g.ldd = ldo;
  g.weights = weights;
  g.w_f32 = w_dtype == TGEMM_DTYPE_F32;
  return finish(tgemm::launch_expert_combine(g, static_cast<hipStream_t>(stream)));
}

int expert_combine_f16_backward(int64_t tokens, int64_t k, int64_t rows, int64_t H, const void* dOUT, int64_t lddo,
                                const void* Y, int64_t ldy, const void* place, const void* weights, int w_dtype, void* dY,
                                int64_t lddy, void* dweights, const void* offsets, int64_t experts, void* stream) {
  const int v = check_rows(tokens, k, rows, H);
  if (v != TGEMM_OK) return v;
  if (((weights != nullptr || dweights != nullptr) && bad_dtype(w_dtype)) || (offsets != nullptr && bad_experts(experts)))
    return TGEMM_EINVAL_DIM;
  const int64_t hmin = at_least_1(H);
  if (lddo < hmin || (dweights != nullptr && ldy < hmin) || (dY != nullptr && lddy < hmin)) return TGEMM_EINVAL_LD;
  const int64_t n = tokens * k;
  if (n == 0 && (dY == nullptr || offsets == nullptr || rows == 0 || H == 0)) return TGEMM_OK;
  if (dY == nullptr && dweights == nullptr) return TGEMM_ENULL;
  if (n > 0 && (place == nullptr || (rows > 0 && H > 0 && (dOUT == nullptr || (dweights != nullptr && Y == nullptr)))))
    return TGEMM_ENULL;
  const unsigned ws = w_dtype == TGEMM_DTYPE_F32 ? 4 : 2;
  if (off(dOUT, 2) || off(Y, 2) || off(dY, 2) || off(place, 4) || off(offsets, 4) || off(weights, ws) || off(dweights, ws))
    return TGEMM_EALIGN;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  ExpertRowsArgs g = rows_args(tokens, k, rows, H, place);
  g.src = halves(dOUT);
  g.lds_ = lddo;
  g.aux = halves(Y);
  g.lda = ldy;
  g.dst = static_cast<_Float16*>(dY);
  g.ldd = lddy;
  g.weights = weights;
  g.dweights = dweights;
  g.w_f32 = w_dtype == TGEMM_DTYPE_F32;
  g.offsets = ints(offsets);
  g.experts = (int)experts;
  return finish(tgemm::launch_expert_combine_grad(g, static_cast<hipStream_t>(stream)));
}

int expert_gemm_f16(int trans_b, int64_t rows, int64_t experts, int64_t N, int64_t K, const void* A, int64_t lda,
                    const void* offsets, const void* B, int64_t ldb, int64_t stride_b, void* C, int64_t ldc, int relu,
                    int zero_rest, void* stream) {
  return run(-1, trans_b ? tgemm::kExpertNT : tgemm::kExpertNN, rows, experts, 0, N, K, A, lda, offsets, B, ldb, stride_b,
             C, ldc, 0, relu, zero_rest, stream);
}

int expert_gemm_f16_cfg(int idx, int trans_b, int64_t rows, int64_t experts, int64_t N, int64_t K, const void* A,
                        int64_t lda, const void* offsets, const void* B, int64_t ldb, int64_t stride_b, void* C,
                        int64_t ldc, int relu, int zero_rest, void* stream) {
  if (idx < 0 || idx >= tgemm::kExpertConfigs) return TGEMM_EINVAL_CFG;
  return run(idx, trans_b ? tgemm::kExpertNT : tgemm::kExpertNN, rows, experts, 0, N, K, A, lda, offsets, B, ldb,
             stride_b, C, ldc, 0, relu, zero_rest, stream);
}

int expert_gemm_f16_tn(int64_t rows, int64_t experts, int64_t M, int64_t N, const void* A, int64_t lda, const void* B,
                       int64_t ldb, const void* offsets, void* C, int64_t ldc, int64_t stride_c, void* stream) {
  return run(-1, tgemm::kExpertTN, rows, experts, M, N, 0, A, lda, offsets, B, ldb, 0, C, ldc, stride_c, 0, 0, stream);
}

int expert_gemm_f16_tn_cfg(int idx, int64_t rows, int64_t experts, int64_t M, int64_t N, const void* A, int64_t lda,
                           const void* B, int64_t ldb, const void* offsets, void* C, int64_t ldc, int64_t stride_c,
                           void* stream) {
  if (idx < 0 || idx >= tgemm::kExpertConfigs) return TGEMM_EINVAL_CFG;
  return run(idx, tgemm::kExpertTN, rows, experts, M, N, 0, A, lda, offsets, B, ldb, 0, C, ldc, stride_c, 0, 0, stream);
}

int expert_gemm_select_config(int form, int64_t rows, int64_t experts, int64_t M, int64_t N, int64_t K, const void* A,
                              int64_t lda, const void* B, int64_t ldb, int64_t stride_b) {
  if (form < tgemm::kExpertNT || form > tgemm::kExpertTN) return TGEMM_EINVAL_CFG;
  const int64_t ldc = at_least_1(N), stride_c = at_least_1(M) * ldc;
  const void* const some = reinterpret_cast<const void*>(256);  // looked at for null and alignment only
  return select(form, rows, experts, M, N, K, A, lda, some, B, ldb, stride_b, some, ldc, stride_c);
}

}  // extern "C"
