// tgemm_expert_gemm.hip -- gfx950 kernels of the experts' products: binary16 operands, float32 sums,
// the rows of each expert given by offsets in device memory.
//
//   rows (NT, NN):  C[p, :] = ReLU?(A[p, :] op(B_e)) for offsets[e] <= p < offsets[e + 1];
//   weights (TN):   C_e = A_e^T B_e, the sum over the expert's rows (zeros for an expert of none).
// Nothing about the groups is known to the host, so a launch of the rows' form has a workgroup for
// every tile that any division of the rows could need (rows / BM + E tile rows); a workgroup finds
// its expert by a sum over the offsets, one lane per 1 / 64 of the experts, and those past the last
// tile leave at once (or zero the rows behind the last group). Offsets are clamped to [0, rows]: no
// value of theirs leads outside the operands.
#include "tgemm_expert.h"
#include "tgemm_pingpong.h"
#include "tgemm_rows.h"

#include <atomic>

namespace tgemm {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));

// Rows [first, first + count) of an expert.
struct RowRange {
  int first, count;
};
__device__ __forceinline__ int clamped(const ExpertGemmArgs& g, int e) {
  const int v = g.offsets[e];
  return v < 0 ? 0 : v < g.rows ? v : g.rows;
}
__device__ __forceinline__ RowRange expert_rows(const ExpertGemmArgs& g, int e) {
  const int a = clamped(g, e), b = clamped(g, e + 1);
  return {a, b > a ? b - a : 0};
}

// A tile of the rows' form.
struct RowTile {
  int e, tm, tn;     // expert, tile inside the expert's part of C
  RowRange rows;
  int past;          // workgroups past the last tile: which one (else -1)
  int past_count;    // how many of them there are
};
// Tile of workgroup blockIdx.x: logical ids (consecutive on an XCD) go through the experts one after
// another, in panels of PANEL tile rows inside an expert, so that neighbours share B's columns.
template <int BM, int PANEL>
__device__ __forceinline__ RowTile find_tile(const ExpertGemmArgs& g, int lane) {
  const int per = (g.experts + 63) / 64, e0 = min(lane * per, g.experts), e1 = min(e0 + per, g.experts);
  int64_t mine = 0;
  for (int e = e0; e < e1; ++e) mine += (expert_rows(g, e).count + BM - 1) / BM;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  const int64_t tile_rows = __shfl(incl, 63, 64), total = tile_rows * g.tiles_n;
  RowTile t;
  if ((int64_t)blockIdx.x >= total) {
    t.past = (int)(blockIdx.x - total);
    t.past_count = (int)(gridDim.x - total);
    t.e = -1;
    return t;
  }
  t.past = -1;
  const int64_t lid = xcd_logical_id(blockIdx.x, total, 1), mt = lid / g.tiles_n;
  const int owner = __builtin_popcountll(__builtin_amdgcn_ballot_w64(incl <= mt));  // lanes whose experts end before mt
  int64_t start = __shfl(incl - mine, owner, 64);
  int e = min(owner * per, g.experts - 1);
  const int last = min(e + per, g.experts) - 1;
  RowRange r = expert_rows(g, e);
  while (e < last && start + (r.count + BM - 1) / BM <= mt) {
    start += (r.count + BM - 1) / BM;
    r = expert_rows(g, ++e);
  }
  int64_t tm, tn;
  const int tiles_m = (r.count + BM - 1) / BM;
  panel_tile(lid - start * g.tiles_n, tiles_m, g.tiles_n, PANEL, &tm, &tn);
  t.e = __builtin_amdgcn_readfirstlane(e);
  t.rows.first = __builtin_amdgcn_readfirstlane(r.first);
  t.rows.count = __builtin_amdgcn_readfirstlane(r.count);
  t.tm = __builtin_amdgcn_readfirstlane((int)tm);
  t.tn = __builtin_amdgcn_readfirstlane((int)tn);
  // (offsets that run backwards or change under the launch could leave no such tile)
  if (t.tm >= tiles_m || t.tn >= g.tiles_n) {
    t.e = -1;
    t.past = 0;
    t.past_count = 0;
  }
  return t;
}

// The rows behind the last group, zeroed by the workgroups past the last tile.
template <int THREADS>
__device__ void zero_rest(const ExpertGemmArgs& g, const RowTile& t) {
  if (!g.zero_rest || t.past_count == 0) return;
  const half8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  const int chunks = (g.N + 7) / 8;
  for (int r = clamped(g, g.experts) + t.past; r < g.rows; r += t.past_count)
    for (int c = threadIdx.x; c < chunks; c += THREADS) store_half8(g.C + (int64_t)r * g.ldc + 8 * c, zero, g.N - 8 * c);
}

// ------------------------------------------------------------------------------------
// BM x BM tiles on the two-group ping-pong schedule (tgemm_pingpong.h): 256 x 256 with k-tiles of
// 32, or 128 x 128 with k-tiles of 64 of which each wave group takes half, the groups' sums joined at
// the end.
template <int BM>
constexpr int kTileKg = BM == 128 ? 2 : 1;
template <int BM>
constexpr int tile_lds_bytes() {
  constexpr int ring = 4 * 2 * BM * 64 * kTileKg<BM>, st = 8 * StagedTile<BM / 2 / kTileKg<BM>, BM * kTileKg<BM> / 4>::BYTES;
  return ring > st ? ring : st;
}
template <bool JOINED, typename A, typename B>
__device__ __forceinline__ auto& pick_sums(A& own, B& joined) {
  if constexpr (JOINED)
    return joined;
  else
    return own;
}

template <int BM, ExpertForm F>
__global__ __launch_bounds__(512) void expert_tiles(ExpertGemmArgs g) {
  constexpr int NW = 8, STAGES = 4, KG = kTileKg<BM>, WN = 4 / KG, BK = 32 * KG;
  constexpr int WTN = BM / WN, FM = BM / 32, FN = WTN / 16;
  constexpr int WTM = BM / 2 / KG, FE = FM / KG;  // after the groups are joined
  constexpr bool A_KMAJ = F != kExpertTN, B_KMAJ = F == kExpertNT;
  using OpA = PpOperand<BM, BK, 16, A_KMAJ, NW>;
  using OpB = PpOperand<BM, BK, 16, B_KMAJ, NW>;
  constexpr int A_BYTES = OpA::BYTES, B_BYTES = OpB::BYTES, PT = OpA::LD + OpB::LD;
  static_assert(OpA::REM == 0 && OpB::REM == 0, "copies split evenly");

  extern __shared__ __attribute__((aligned(16))) char smem[];
  char* const a_lds = smem;
  char* const b_lds = smem + STAGES * A_BYTES;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  int row0, col0, mvalid, K;
  const _Float16 *A, *B;
  _Float16* C;
  if constexpr (F == kExpertTN) {
    const int tiles = g.tiles_m * g.tiles_n;
    const int64_t lid = xcd_logical_id(blockIdx.x, (int64_t)tiles * g.experts, 1);
    const int e = __builtin_amdgcn_readfirstlane((int)(lid / tiles));
    int64_t tm, tn;
    panel_tile(lid - (int64_t)e * tiles, g.tiles_m, g.tiles_n, 4, &tm, &tn);
    const RowRange r = expert_rows(g, e);
    row0 = __builtin_amdgcn_readfirstlane((int)tm) * BM;
    col0 = __builtin_amdgcn_readfirstlane((int)tn) * BM;
    mvalid = min(BM, g.M - row0);
    K = __builtin_amdgcn_readfirstlane(r.count);
    const int64_t first = __builtin_amdgcn_readfirstlane(r.first);
    A = g.A + first * g.lda;
    B = g.B + first * g.ldb;
    C = g.C + e * g.stride_c;
  } else {
    const RowTile t = find_tile<BM, 4>(g, lane);
    if (t.e < 0) return zero_rest<512>(g, t);
    row0 = t.tm * BM;
    col0 = t.tn * BM;
    mvalid = min(BM, t.rows.count - row0);
    K = g.K;
    A = g.A + (int64_t)t.rows.first * g.lda;
    B = g.B + t.e * g.stride_b;
    C = g.C + (int64_t)t.rows.first * g.ldc;
  }
  const int nvalid = min(BM, g.N - col0);
  const int nk = (K + BK - 1) / BK, kin_last = K - (nk - 1) * BK;

  OpA opa;
  OpB opb;
  opa.init_copies(A, g.lda, row0, mvalid, kin_last, wave, lane);
  opb.init_copies(B, g.ldb, col0, nvalid, kin_last, wave, lane);
  const uint32_t a_lds0 = lds_addr(a_lds) + wave * 1024, b_lds0 = lds_addr(b_lds) + wave * 1024;
  TileStream sa, sb;
  sa.init(opa, nk);
  sb.init(opb, nk);
  auto copy_tile = [&](int kt, auto) __attribute__((always_inline)) {
    const bool last = sa.at_last();
    const int4v ra = sa.next(), rb = sb.next();
    const int slot = kt % STAGES;
#pragma unroll
    for (int j = 0; j < OpA::LD; ++j)
      dma_to_lds(ra, a_lds0 + slot * A_BYTES + j * NW * 1024, last ? opa.off_last[j] : opa.off[j]);
#pragma unroll
    for (int j = 0; j < OpB::LD; ++j)
      dma_to_lds(rb, b_lds0 + slot * B_BYTES + j * NW * 1024, last ? opb.off_last[j] : opb.off[j]);
  };
  const int kg = KG == 2 ? wave >> 2 : 0, wv = wave % (2 * WN), wm = wv / WN, wn = wv % WN;
  opa.init_frags(wm * (BM / 2), lane);
  opb.init_frags(wn * WTN, lane);
  half8 fa[FM], fb[FN];
  auto read_tile = [&](int kt) __attribute__((always_inline)) {
    const char* const As = a_lds + (kt % STAGES) * A_BYTES;
    const char* const Bs = b_lds + (kt % STAGES) * B_BYTES;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) fa[fm] = opa.frag(As, fm, kg);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) fb[fn] = opb.frag(Bs, fn, kg);
  };
  float4v sum[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sum[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  auto mma_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        sum[fm][fn] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[fn], fa[fm], sum[fm][fn], 0, 0, 0);
  };
  pingpong_schedule<STAGES, PT, PT, (A_KMAJ && B_KMAJ && BM == 256)>(wave / 4, nk, copy_tile, read_tile, mma_tile);
  __syncthreads();  // the ring is free for staging
  float4v joined_sum[KG == 2 ? FE : 1][FN];
  if constexpr (KG == 2) join_k_groups<FM, FN>(smem, sum, joined_sum, wave, lane);
  float4v(&acc)[FE][FN] = pick_sums<KG == 2>(sum, joined_sum);

  const int wr0 = wm * (BM / 2) + kg * WTM, wc0 = wn * WTN;
  using ST = StagedTile<WTM, WTN>;
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  store_staged<ST, WTM, false>(stage, lane, C + (int64_t)(row0 + wr0) * g.ldc + col0 + wc0, g.ldc, mvalid - wr0,
                               nvalid - wc0, g.vec_c);
}

// ------------------------------------------------------------------------------------
// Few rows an expert: 32 x 128 tiles, four waves of 32 columns, k-tiles of 64 through a ring of
// kStages slots, one barrier each: after the barrier of tile t the copies of tile t + kStages - 1 go
// into the slot of tile t - 1, which every wave has read. Bound by reading the weights of the
// experts that are met.
constexpr int kSmallStages = 4;
template <ExpertForm F>
struct SmallTile {
  static constexpr int BM = 32, BN = 128, BK = 64, NW = 4;
  using OpA = PpOperand<BM, BK, 16, true, NW>;
  using OpB = PpOperand<BN, BK, 16, F == kExpertNT, NW>;
  static constexpr int PT = OpA::LD + OpB::LD, SLOT = OpA::BYTES + OpB::BYTES, LDS = kSmallStages * SLOT;
  static_assert(OpA::REM == 0 && OpB::REM == 0, "copies split evenly");
};

template <ExpertForm F>
__global__ __launch_bounds__(256) void expert_small(ExpertGemmArgs g) {
  using T = SmallTile<F>;
  using OpA = typename T::OpA;
  using OpB = typename T::OpB;
  constexpr int BM = T::BM, BN = T::BN, BK = T::BK, NW = T::NW, STAGES = kSmallStages;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const RowTile t = find_tile<BM, 4>(g, lane);
  if (t.e < 0) return zero_rest<256>(g, t);
  const int row0 = t.tm * BM, col0 = t.tn * BN;
  const int mvalid = min(BM, t.rows.count - row0), nvalid = min(BN, g.N - col0);
  const int nk = (g.K + BK - 1) / BK, kin_last = g.K - (nk - 1) * BK;
  OpA opa;
  OpB opb;
  opa.init_copies(g.A + (int64_t)t.rows.first * g.lda, g.lda, row0, mvalid, kin_last, wave, lane);
  opb.init_copies(g.B + t.e * g.stride_b, g.ldb, col0, nvalid, kin_last, wave, lane);
  const uint32_t a_lds0 = lds_addr(smem) + wave * 1024, b_lds0 = a_lds0 + OpA::BYTES;
  TileStream sa, sb;
  sa.init(opa, nk);
  sb.init(opb, nk);
  auto copy_tile = [&](int kt) __attribute__((always_inline)) {
    const bool last = sa.at_last();
    const int4v ra = sa.next(), rb = sb.next();
    const int slot = kt % STAGES;
#pragma unroll
    for (int j = 0; j < OpA::LD; ++j)
      dma_to_lds(ra, a_lds0 + slot * T::SLOT + j * NW * 1024, last ? opa.off_last[j] : opa.off[j]);
#pragma unroll
    for (int j = 0; j < OpB::LD; ++j)
      dma_to_lds(rb, b_lds0 + slot * T::SLOT + j * NW * 1024, last ? opb.off_last[j] : opb.off[j]);
  };
  opa.init_frags(0, lane);
  opb.init_frags(wave * 32, lane);
  float4v acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) copy_tile(i);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vmcnt<T::PT * (STAGES - 2)>();  // this thread's copies of tile kt have landed
    lds_barrier();                        // everyone's have, and tile kt - 1 is read
    copy_tile(kt + STAGES - 1);
    const char* const As = smem + (kt % STAGES) * T::SLOT;
    const char* const Bs = As + OpA::BYTES;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      half8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = opa.frag(As, i, ks);
        fb[i] = opb.frag(Bs, i, ks);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  wait_vmcnt<0>();
  __syncthreads();  // the ring is free for staging
  using ST = StagedTile<32, 32>;
  static_assert(NW * ST::BYTES <= T::LDS, "staged tiles");
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  store_staged<ST, 32, false>(stage, lane, g.C + (int64_t)(t.rows.first + row0) * g.ldc + col0 + wave * 32, g.ldc, mvalid,
                              nvalid - wave * 32, g.vec_c);
}

// ------------------------------------------------------------------------------------
// Any alignment, stride and size: 128 x 128 tiles, four waves of 64 x 64, 32 k at a time through a
// double-buffered LDS tile filled through registers.
template <ExpertForm F>
__global__ __launch_bounds__(256) void expert_generic(ExpertGemmArgs g) {
  constexpr int BM = 128, ROW = 40;  // halves per LDS row: 16-byte aligned, rows spread over the banks
  __shared__ __attribute__((aligned(16))) _Float16 at[2][BM * ROW], bt[2][BM * ROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64, lrow = lane & 15, lkg = lane >> 4;
  int row0, col0, mvalid, K;
  const _Float16 *A, *B;
  _Float16* C;
  if constexpr (F == kExpertTN) {
    const int tiles = g.tiles_m * g.tiles_n, e = (int)(blockIdx.x / tiles), t = (int)(blockIdx.x % tiles);
    const RowRange r = expert_rows(g, e);
    row0 = t / g.tiles_n * BM;
    col0 = t % g.tiles_n * BM;
    mvalid = g.M - row0;
    K = r.count;
    A = g.A + (int64_t)r.first * g.lda;
    B = g.B + (int64_t)r.first * g.ldb;
    C = g.C + e * g.stride_c;
  } else {
    const RowTile t = find_tile<BM, 4>(g, lane);
    if (t.e < 0) return zero_rest<256>(g, t);
    row0 = t.tm * BM;
    col0 = t.tn * BM;
    mvalid = t.rows.count - row0;
    K = g.K;
    A = g.A + (int64_t)t.rows.first * g.lda;
    B = g.B + t.e * g.stride_b;
    C = g.C + (int64_t)t.rows.first * g.ldc;
  }
  const int nvalid = g.N - col0;
  // An operand's tile, two chunks of eight values a thread: along k of row tid / 2 where k is
  // contiguous, else along the rows of k = (2 tid + h) / 16.
  half8 av[2], bv[2];
  auto fetch = [&](auto kmaj, const _Float16* X, int64_t ld, int r0, int valid, int kt, half8 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (decltype(kmaj)::value) {
        const int r = tid >> 1, k = 32 * kt + 16 * (tid & 1) + 8 * h;
        v[h] = load_half8(X + (int64_t)(r0 + r) * ld + k, r < valid ? K - k : 0);
      } else {
        const int u = 2 * tid + h, k = 32 * kt + u / 16, r = 8 * (u % 16);
        v[h] = load_half8(X + (int64_t)k * ld + r0 + r, k < K ? valid - r : 0);
      }
    }
  };
  auto put = [&](auto kmaj, _Float16* tile, const half8 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (decltype(kmaj)::value) {
        *(half8*)&tile[(tid >> 1) * ROW + 16 * (tid & 1) + 8 * h] = v[h];
      } else {
        const int u = 2 * tid + h;
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[(8 * (u % 16) + e) * ROW + u / 16] = v[h][e];
      }
    }
  };
  using KA = std::integral_constant<bool, F != kExpertTN>;
  using KB = std::integral_constant<bool, F == kExpertNT>;
  float4v acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  const int nk = (K + 31) / 32;
  if (nk > 0) {
    fetch(KA{}, A, g.lda, row0, mvalid, 0, av);
    fetch(KB{}, B, g.ldb, col0, nvalid, 0, bv);
    put(KA{}, at[0], av);
    put(KB{}, bt[0], bv);
  }
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int buf = kt & 1;
    if (kt + 1 < nk) {
      fetch(KA{}, A, g.lda, row0, mvalid, kt + 1, av);
      fetch(KB{}, B, g.ldb, col0, nvalid, kt + 1, bv);
    }
    half8 fa[4], fb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa[f] = *(const half8*)&at[buf][(wm + 16 * f + lrow) * ROW + 8 * lkg];
      fb[f] = *(const half8*)&bt[buf][(wn + 16 * f + lrow) * ROW + 8 * lkg];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    if (kt + 1 < nk) {
      put(KA{}, at[buf ^ 1], av);
      put(KB{}, bt[buf ^ 1], bv);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = wm + 16 * i + lrow;
    if (m >= mvalid) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = wn + 16 * j + 4 * lkg + e;
        if (c < nvalid)
          C[(int64_t)(row0 + m) * g.ldc + col0 + c] = (_Float16)(g.relu ? relu_f(acc[i][j][e]) : acc[i][j][e]);
      }
  }
}

// A kernel with more than the default dynamic LDS: the limit is raised once per kernel and device.
template <typename K>
hipError_t launch(K kern, int threads, int lds, std::atomic<uint64_t>& ready, const ExpertGemmArgs& g, unsigned grid,
                  hipStream_t s, int device) {
  const uint64_t bit = 1ull << (device & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), lds, s, g);
  return hipGetLastError();
}
template <int BM, ExpertForm F>
hipError_t launch_tiles(const ExpertGemmArgs& g, unsigned grid, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  return launch(expert_tiles<BM, F>, 512, tile_lds_bytes<BM>(), ready, g, grid, s, device);
}
template <ExpertForm F>
hipError_t launch_form(int cfg, const ExpertGemmArgs& g, unsigned grid, hipStream_t s, int device) {
  switch (cfg) {
    case kExpert256: return launch_tiles<256, F>(g, grid, s, device);
    case kExpert128: return launch_tiles<128, F>(g, grid, s, device);
    case kExpert32:
      if constexpr (F != kExpertTN) {
        static std::atomic<uint64_t> ready{0};
        return launch(expert_small<F>, 256, SmallTile<F>::LDS, ready, g, grid, s, device);
      } else {
        return hipErrorNotSupported;
      }
    default:
      hipLaunchKernelGGL(expert_generic<F>, dim3(grid), dim3(256), 0, s, g);
      return hipGetLastError();
  }
}

}  // namespace

hipError_t launch_expert_gemm(int cfg, ExpertForm form, const ExpertGemmArgs& args, hipStream_t s, int device) {
  ExpertGemmArgs g = args;
  const int64_t grid = expert_gemm_groups(cfg, form, g.rows, g.experts, g.M, g.N);
  g.tiles_m = form == kExpertTN ? (int)ceil_div(g.M, expert_tile_m(cfg)) : 0;
  g.tiles_n = (int)ceil_div(g.N, expert_tile_n(cfg));
  if (form == kExpertNT) return launch_form<kExpertNT>(cfg, g, (unsigned)grid, s, device);
  if (form == kExpertNN) return launch_form<kExpertNN>(cfg, g, (unsigned)grid, s, device);
  return launch_form<kExpertTN>(cfg, g, (unsigned)grid, s, device);
}

}  // namespace tgemm
