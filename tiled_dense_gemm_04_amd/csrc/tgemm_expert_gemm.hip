// tgemm_expert_gemm.hip -- gfx950 kernels of the experts' products: binary16 operands, float32 sums,
// the rows of each expert given by offsets in device memory.
//
//   rows (NT, NN):  C[p, :] = ReLU?(A[p, :] op(B_e)) for offsets[e] <= p < offsets[e + 1];
//   weights (TN):   C_e = A_e^T B_e, the sum over the expert's rows (zeros for an expert of none).
// Nothing about the groups is known to the host. The tile kernels run one workgroup a compute unit, each
// of which finds the tiles it goes over from the offsets (expert_tiles, expert_tiles_weights); the ones
// for few rows have a workgroup for every tile that any division of the rows could need, and those
// past the last tile leave at once (or zero the rows behind the last group). Offsets are clamped to [0,
// rows]: no value of theirs leads outside the operands.
// What bounds them: the binary16 MFMAs at their power limit and the rounds of tiles (uneven experts, 16384
// rows on 16 of them, 4096 x 2048: rows' form 281 to 304 us with B N x K, by the box, and 266 with K x N, weights'
// form 281 to 284, of 275 GFLOP; one expert 264, the dense kernel of this library 271); with few rows an expert, reading the
// weights (64 rows on 64 experts of 2048 x 4096, about 36 of them met: 109 us, 5.5 TB/s).
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

// The rows behind the last group, zeroed by `parts` workgroups, of which this is `part`.
template <int THREADS>
__device__ void zero_rest(const ExpertGemmArgs& g, int part, int parts) {
  if (!g.zero_rest || parts == 0) return;
  const half8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  const uint32_t chunks = ((uint32_t)g.N + 7) / 8;
  every_nth_row(clamped(g, g.experts) + (int64_t)part, g.rows, parts, [&](int64_t r) {
    for (uint32_t c = threadIdx.x; c < chunks; c += THREADS) store_half8(g.C + r * g.ldc + 8 * c, zero, g.N - 8 * (int)c);
  });
}

// ------------------------------------------------------------------------------------
// BM x BN tiles on the two-group ping-pong schedule (tgemm_pingpong.h): 256 x 256 with k-tiles of
// 32, or 128 x 128 and 64 x 128 with k-tiles of 64 of which each wave group takes half, the groups' sums
// joined at the end. A, B and C point at the tile's first row or column of each.
template <int BM>
constexpr int kTileKg = BM == 256 ? 1 : 2;
template <int BM>
constexpr int tile_lds_bytes() {
  constexpr int ring = 4 * 2 * BM * 64 * kTileKg<BM>, st = 8 * StagedTile<BM / 2 / kTileKg<BM>, BM * kTileKg<BM> / 4>::BYTES;
  return ring > st ? ring : st;
}
constexpr int kTileLds = tile_lds_bytes<256>() > tile_lds_bytes<128>() ? tile_lds_bytes<256>() : tile_lds_bytes<128>();
template <bool JOINED, typename A, typename B>
__device__ __forceinline__ auto& pick_sums(A& own, B& joined) {
  if constexpr (JOINED)
    return joined;
  else
    return own;
}

template <int BM, int BN, ExpertForm F>
__device__ __forceinline__ void tile_product(const ExpertGemmArgs& g, char* smem, const _Float16* A, const _Float16* B,
                                             _Float16* C, int mvalid, int nvalid, int K) {
  constexpr int NW = 8, STAGES = 4, KG = kTileKg<BM>, WN = 4 / KG, BK = 32 * KG;
  constexpr int WTN = BN / WN, FM = BM / 32, FN = WTN / 16;
  constexpr int WTM = BM / 2 / KG, FE = FM / KG;  // after the groups are joined
  constexpr bool A_KMAJ = F != kExpertTN, B_KMAJ = F == kExpertNT;
  using OpA = PpOperand<BM, BK, 16, A_KMAJ, NW>;
  using OpB = PpOperand<BN, BK, 16, B_KMAJ, NW>;
  constexpr int A_BYTES = OpA::BYTES, B_BYTES = OpB::BYTES, PT = OpA::LD + OpB::LD;
  static_assert(OpA::REM == 0 && OpB::REM == 0, "copies split evenly");

  char* const a_lds = smem;
  char* const b_lds = smem + STAGES * A_BYTES;
  // (a thread index of the tile's own: what follows from it is not carried over the loop over tiles,
  // where it would spill)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  mvalid = min(BM, mvalid);
  nvalid = min(BN, nvalid);
  const int nk = k_tiles(K, BK), kin_last = K - (nk - 1) * BK;

  OpA opa;
  OpB opb;
  opa.init_copies(A, g.lda, 0, mvalid, kin_last, wave, lane);
  opb.init_copies(B, g.ldb, 0, nvalid, kin_last, wave, lane);
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
  store_staged<ST, WTM, false>(stage, lane, C + (int64_t)wr0 * g.ldc + wc0, g.ldc, mvalid - wr0, nvalid - wc0, g.vec_c);
}

// How an M x N part of C is cut: 256 x 256 tiles, and 128 x 128 ones along its lower and right edge
// where no more than half of a big tile would be used.
struct Cut {
  uint32_t mb, nb;           // big tiles
  uint32_t low, low_count;   // first row of the lower edge, its tiles (0: none)
  uint32_t right_count;      // tiles of the right edge (at column 256 nb)
  __device__ Cut(uint32_t M, uint32_t N) {
    mb = (M + 127) / 256;
    nb = (N + 127) / 256;
    low = mb * 256;
    low_count = M > low ? (N + 127) / 128 : 0;
    right_count = N > nb * 256 ? (min(M, low) + 127) / 128 : 0;
  }
  __device__ uint32_t big() const { return mb * nb; }
  __device__ uint32_t small() const { return low_count + right_count; }
};

// The tiles of the rows' form, in the order in which its workgroups take them (workgroup w those at w,
// w + gridDim.x, ...): `kept` big tiles; the other big ones in quarters; the small ones. One big tile
// takes about as long as three small ones, so big tiles that would fill less than half of the compute
// units in a last round go in quarters; and the small ones that would fill no more than half of them
// in a last round go in halves, 64 x 128, which take two thirds to four fifths of a small one's time
// (4096 rows, 8 experts, 4096 x 2048: 88 to 85 us; 8190, 2048 x 1032: 55 to 52.5; 300 rows, one of 4096 x
// 4096: 30 to 26). (Counts are of 32 bits: the host keeps those of offsets that do not decrease below
// 2^31, and the length of the list below that bound whatever the offsets hold.)
struct TileList {
  uint32_t kept, quarters, edges;  // big tiles, quarters (4 a tile), edge tiles
  uint32_t halved;                 // of the last two, the ones that go in halves
  __device__ void cut(uint32_t big, uint32_t small, int mode) {
    constexpr uint32_t G = kExpertTileGroups;
    const uint32_t rest = big % G;
    bool keep = mode == kTilesBig;
    if (mode == kTilesAuto) {
      const uint32_t idle = rest == 0 ? 0 : G - rest;
      const uint32_t as_big = (rest == 0 ? 0 : 3) + (small > idle ? (small - idle + G - 1) / G : 0);
      keep = as_big <= (4 * rest + small + G - 1) / G;
    }
    kept = mode == kTilesSmall ? 0 : keep ? big : big - rest;
    quarters = 4 * (big - kept);
    edges = small;
    const uint32_t last = (quarters + edges) % G;
    halved = mode == kTilesAuto && kept % G == 0 && last <= G / 2 ? last : 0;
  }
};

// A tile: of which expert, from which row and column of its part of C on.
struct Tile {
  int e;
  uint32_t row0, col0;
  RowRange rows;
  int size;  // its rows: 256, 128 or 64 (of 128 columns)
  // tile i of the big ones (or quarter 0 .. 3 of it) or of the small ones of a part cut by c
  __device__ void place(const Cut& c, uint32_t i, bool of_big, uint32_t quarter) {
    if (of_big) {  // panels of four tile rows, the tile rows of a panel first
      const uint32_t per_panel = 4 * c.nb, p = i / per_panel, within = i - p * per_panel, height = min(c.mb - 4 * p, 4u);
      const uint32_t tn = within / height, tm = 4 * p + within - tn * height;
      row0 = tm * 256 + (quarter < 4 ? 128 * (quarter >> 1) : 0);
      col0 = tn * 256 + (quarter < 4 ? 128 * (quarter & 1) : 0);
    } else {
      const bool lower = i < c.low_count;
      row0 = lower ? c.low : 128 * (i - c.low_count);
      col0 = lower ? 128 * i : 256 * c.nb;
    }
    size = of_big && quarter == 4 ? 256 : 128;
  }
  __device__ void make_uniform() {
    e = __builtin_amdgcn_readfirstlane(e);
    rows.first = __builtin_amdgcn_readfirstlane(rows.first);
    rows.count = __builtin_amdgcn_readfirstlane(rows.count);
    row0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)row0);
    col0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)col0);
  }
};

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// Consecutive ids of `total` on one XCD (xcd_logical_id in 32 bits), inside each round of the launch's
// workgroups: an XCD that took a contiguous part of all of them would take the longest of the
// weights' form, which come first (16384 rows, 16 uneven experts, 4096 x 2048: 495 us, so 281).
__device__ __forceinline__ uint32_t xcd_id(uint32_t at, uint32_t total) {
  constexpr uint32_t G = kExpertTileGroups;
  const uint32_t first = at / G * G, wg = at - first, n = min(G, total - first);
  if (n < (uint32_t)kNumXcd) return at;
  const uint32_t q = n / kNumXcd, r = n % kNumXcd, x = wg % kNumXcd, j = wg / kNumXcd;
  return first + x * q + min(x, r) + j;
}

// The rows' form: the list and what finds a tile in it, in LDS (the registers are the product's).
struct TileFinder {
  TileList list;
  uint32_t big_incl[64], small_incl[64];  // tiles of a lane's experts and those before
  int offsets[kMaxExperts + 1];           // clamped
};
__device__ __forceinline__ RowRange rows_of(const TG_LDS TileFinder* f, int e) {
  const int a = f->offsets[e], b = f->offsets[e + 1];
  return {a, b > a ? b - a : 0};
}

// By the whole workgroup (a barrier follows).
__device__ __forceinline__ void init_finder(const ExpertGemmArgs& g, TG_LDS TileFinder* f) {
  for (int e = threadIdx.x; e <= g.experts; e += 512) f->offsets[e] = clamped(g, e);
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x;
  const int per = (g.experts + 63) / 64, e0 = min(lane * per, g.experts), e1 = min(e0 + per, g.experts);
  uint32_t big = 0, small = 0;
  for (int e = e0; e < e1; ++e) {
    const Cut c(rows_of(f, e).count, g.N);
    big += c.big();
    small += c.small();
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t b = __shfl_up(big, o, 64), s = __shfl_up(small, o, 64);
    if (lane >= o) {
      big += b;
      small += s;
    }
  }
  f->big_incl[lane] = big;
  f->small_incl[lane] = small;
  TileList list;
  list.cut(__shfl(big, 63, 64), __shfl(small, 63, 64), g.mode);
  if (lane == 0) {
    f->list.kept = list.kept;
    f->list.quarters = list.quarters;
    f->list.edges = list.edges;
    f->list.halved = list.halved;
  }
}

// Tile `at` of the list into t (uniform); false past its end.
__device__ __forceinline__ bool find_in_rows(const ExpertGemmArgs& g, const TG_LDS TileFinder* f, uint32_t at, int lane, Tile& t) {
  const uint32_t kept = uniform(f->list.kept), quarters = uniform(f->list.quarters), halved = uniform(f->list.halved);
  const uint32_t rest = quarters + uniform(f->list.edges) - halved;
  if (at >= min(kept + rest + 2 * halved, g.max_tiles)) return false;
  // i: which of the big tiles, or of the small ones; a quarter names its big tile
  uint32_t i, quarter = 4, half = 2;
  bool big = true;
  if (at < kept) {
    i = xcd_id(at, kept);
  } else {
    if (at < kept + rest) {
      i = xcd_id(at - kept, rest);
    } else {
      i = xcd_id(at - kept - rest, 2 * halved);
      half = i & 1;
      i = rest + i / 2;
    }
    big = i < quarters;
    if (big) {
      quarter = i & 3;
      i = kept + i / 4;
    } else {
      i -= quarters;
    }
  }
  const TG_LDS uint32_t* const incl = big ? f->big_incl : f->small_incl;
  const int per = (g.experts + 63) / 64;
  const int owner = __builtin_popcountll(__builtin_amdgcn_ballot_w64(incl[lane] <= i));  // lanes whose tiles end before i
  if (owner > 0) i -= uniform(incl[owner - 1]);
  t.e = min(owner * per, g.experts - 1);
  const int last = min(t.e + per, g.experts) - 1;
  for (;;) {
    t.rows = rows_of(f, t.e);
    const Cut c(t.rows.count, g.N);
    const uint32_t n = big ? c.big() : c.small();
    if (i < n || t.e == last) {
      t.place(c, i, big, quarter);
      break;
    }
    i -= n;
    ++t.e;
  }
  if (half < 2) {
    t.row0 += 64 * half;
    t.size = 64;
  }
  t.make_uniform();
  return true;
}

template <ExpertForm F>
__global__ __launch_bounds__(512) void expert_tiles(ExpertGemmArgs args) {
  static_assert(F != kExpertTN, "the rows' form");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63;
  TG_LDS TileFinder* const finder = (TG_LDS TileFinder*)(smem + kTileLds);
  init_finder(args, finder);
  // The arguments are read again for every tile: kept over the loop they would spill.
  typedef const __attribute__((address_space(4))) ExpertGemmArgs KernelArgs;
  KernelArgs* source = (KernelArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  for (uint32_t at = blockIdx.x;; at += gridDim.x) {
    asm volatile("" : "+s"(source));
    ExpertGemmArgs g;
    __builtin_memcpy(&g, (const void*)source, sizeof(g));
    __syncthreads();  // the list is there, and every wave has stored its part of the tile before
    Tile t;
    if (!find_in_rows(g, finder, at, lane, t)) break;
    // (a quarter or a half past the edge; offsets that run backwards can leave no such tile)
    if (t.row0 >= (uint32_t)t.rows.count || t.col0 >= (uint32_t)g.N) continue;
    const int64_t first = (int64_t)t.rows.first + t.row0;
    const _Float16* const A = g.A + first * g.lda;
    const _Float16* const B = g.B + t.e * g.stride_b + (F == kExpertNT ? (int64_t)t.col0 * g.ldb : t.col0);
    _Float16* const C = g.C + first * g.ldc + t.col0;
    if (t.size == 256)
      tile_product<256, 256, F>(g, smem, A, B, C, t.rows.count - t.row0, g.N - t.col0, g.K);
    else if (t.size == 64)
      tile_product<64, 128, F>(g, smem, A, B, C, t.rows.count - t.row0, g.N - t.col0, g.K);
    else
      tile_product<128, 128, F>(g, smem, A, B, C, t.rows.count - t.row0, g.N - t.col0, g.K);
  }
  zero_rest<512>(args, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------------------------
// The weights' form. Every expert has the same tiles, each as long as the expert has rows, so the tiles
// are taken in the order of their time, forth and back over the workgroups (those that had a long tile
// in one round have a short one in the next), and the big ones of the `q` experts of most rows go in
// quarters. In units of a row of a big tile, a big tile of K rows takes K + 170 and a small one 0.3 K +
// 170 (measured: 4 us and 0.024 a row, 4 us and 0.0072 a row); q is what makes least the tiles' time spread
// over the compute units plus half of the longest one's. (A workgroup per tile, which the hardware
// hands to the next free compute unit, costs 5 us more a tile: 16384 rows, 16 experts, 2048 x 1024: 99 to
// 123 us.) More than 64 experts, which one lane each cannot rank, are taken as they come, in big tiles: equal
// experts lose little by it (16384 rows, 2048 x 1024: 64 of them 118 us, 65 124), uneven ones a fifth to a third
// (134 and 161; 1024 x 512: 40 and 55), 128 of them 213 us where their bytes take 123.
struct WeightTiles {
  uint32_t total, q;
  int expert[64];                                      // of rank r, most rows first
  uint32_t big_at[64], bigs[64], small_at[64], smalls[64];  // where its tiles come in the list
};
// By the first wave (a barrier follows).
__device__ __forceinline__ void init_weights(const ExpertGemmArgs& g, TG_LDS WeightTiles* f, int lane) {
  const Cut c(g.M, g.N);
  const uint32_t B = c.big(), S = c.small(), E = g.experts;
  if (E > 64) {
    if (lane == 0) f->total = E * ((g.mode == kTilesSmall ? 4 * B : B) + S);
    return;
  }
  const bool real = lane < (int)E;
  const int mine = real ? expert_rows(g, lane).count : -1;
  uint32_t rank = 0;
  for (uint32_t j = 0; j < E; ++j) {
    const int other = __builtin_amdgcn_readlane(mine, (int)j);
    rank += other > mine || (other == mine && (int)j < lane) ? 1 : 0;
  }
  if (!real) rank = lane;
  f->expert[rank] = lane;
  // lane r: the rows of the r-th longest expert
  const float K = (float)max(__builtin_amdgcn_ds_permute((int)rank * 4, mine), 0);
  uint32_t q = g.mode == kTilesSmall ? E : 0;
  if (g.mode == kTilesAuto) {
    float longer = K;  // rows of those longer
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const float up = __shfl_up(longer, o, 64);
      if (lane >= o) longer += up;
    }
    const float all = __shfl(longer, 63, 64), top = __shfl(K, 0, 64), n = (float)lane;
    longer -= K;
    // lane r prices q = r
    const float spread = (B * (all - longer + 170.0f * (E - n)) + 4 * B * (0.3f * longer + 170.0f * n) +
                          S * (0.3f * all + 170.0f * E)) * (1.0f / kExpertTileGroups);
    const float longest = fmaxf(real ? K + 170.0f : 0.0f, lane > 0 || S > 0 ? 0.3f * top + 170.0f : 0.0f);
    const float cost = lane > (int)E ? __builtin_inff() : spread + 0.5f * longest;
    float least = cost;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) least = fminf(least, __shfl_xor(least, o, 64));
    q = min((uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(cost == least) | 1ull << 63), E);
  }
  // Big and small tiles each lie in the order of their time, rank by rank: where a rank's come among
  // those of the other kind is a search.
  const float big_time = K + 170.0f, small_time = 0.3f * K + 170.0f;
  auto bigs_before = [&](uint32_t r) { return r > q ? (r - q) * B : 0; };   // of the ranks below r
  auto smalls_before = [&](uint32_t r) { return 4 * B * min(r, q) + S * r; };
  uint32_t smalls_longer = 0, bigs_longer = 0;  // ranks whose small (big) tiles come before this one's big (small)
  for (int step = 32, last = 0; last < 2; last += step == 1, step = step > 1 ? step / 2 : 1) {
    const uint32_t a = smalls_longer + step - 1, b = bigs_longer + step - 1;
    const float ta = __shfl(small_time, (int)(a & 63), 64), tb = __shfl(big_time, (int)(b & 63), 64);
    smalls_longer += a < E && ta > big_time ? step : 0;
    bigs_longer += b < E && tb >= small_time ? step : 0;
  }
  f->big_at[lane] = bigs_before(lane) + smalls_before(smalls_longer);
  f->bigs[lane] = real && (uint32_t)lane >= q ? B : 0;
  f->small_at[lane] = smalls_before(lane) + bigs_before(bigs_longer);
  f->smalls[lane] = real ? ((uint32_t)lane < q ? 4 * B : 0) + S : 0;
  if (lane == 0) {
    f->total = bigs_before(E) + smalls_before(E);
    f->q = q;
  }
}

// The tile of workgroup blockIdx.x in round `round` into t (uniform); false past the last.
__device__ __forceinline__ bool find_in_weights(const ExpertGemmArgs& g, const TG_LDS WeightTiles* f, uint32_t round, int lane,
                                                Tile& t) {
  constexpr uint32_t G = kExpertTileGroups;
  const Cut c(g.M, g.N);
  const uint32_t B = c.big(), S = c.small(), total = uniform(f->total), first = round * G;
  if (first + blockIdx.x >= total) return false;
  uint32_t at = xcd_id(first + blockIdx.x, total);
  if (round & 1) at = first + min(G, total - first) - 1 - (at - first);
  uint32_t i, quarter = 4, quarters;  // quarters of the tile's expert
  bool of_big;
  if (g.experts > 64) {
    quarters = g.mode == kTilesSmall ? 4 * B : 0;
    const uint32_t each = (quarters > 0 ? quarters : B) + S;
    t.e = (int)(at / each);
    i = at - t.e * each;
    of_big = quarters == 0 && i < B;
    if (quarters == 0 && !of_big) i -= B;
  } else {
    const uint32_t big_at = f->big_at[lane], small_at = f->small_at[lane];
    const uint64_t in_big = __builtin_amdgcn_ballot_w64(at - big_at < f->bigs[lane]);  // (unsigned: from its start on)
    const uint64_t in_small = __builtin_amdgcn_ballot_w64(at - small_at < f->smalls[lane]);
    of_big = in_big != 0;
    const int r = (int)__builtin_ctzll((of_big ? in_big : in_small) | 1ull << 63);
    i = at - (uint32_t)__builtin_amdgcn_readlane((int)(of_big ? big_at : small_at), r);
    quarters = (uint32_t)r < uniform(f->q) ? 4 * B : 0;
    t.e = f->expert[r];
  }
  if (!of_big) {
    of_big = i < quarters;
    if (of_big) {
      quarter = i & 3;
      i /= 4;
    } else {
      i -= quarters;
    }
  }
  t.e = min(t.e, g.experts - 1);
  t.rows = expert_rows(g, t.e);
  t.place(c, i, of_big, quarter);
  t.make_uniform();
  return true;
}

__global__ __launch_bounds__(512) void expert_tiles_weights(ExpertGemmArgs args) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63;
  TG_LDS WeightTiles* const tiles = (TG_LDS WeightTiles*)(smem + kTileLds);
  if (threadIdx.x < 64) init_weights(args, tiles, lane);
  typedef const __attribute__((address_space(4))) ExpertGemmArgs KernelArgs;  // (as in expert_tiles)
  KernelArgs* source = (KernelArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  for (uint32_t round = 0;; ++round) {
    asm volatile("" : "+s"(source));
    ExpertGemmArgs g;
    __builtin_memcpy(&g, (const void*)source, sizeof(g));
    __syncthreads();  // the list is there, and every wave has stored its part of the tile before
    Tile t;
    if (!find_in_weights(g, tiles, round, lane, t)) break;
    const int64_t first = t.rows.first;
    const _Float16* const A = g.A + first * g.lda + t.row0;
    const _Float16* const B = g.B + first * g.ldb + t.col0;
    _Float16* const C = g.C + t.e * g.stride_c + (int64_t)t.row0 * g.ldc + t.col0;
    if (t.size == 256)
      tile_product<256, 256, kExpertTN>(g, smem, A, B, C, g.M - t.row0, g.N - t.col0, t.rows.count);
    else
      tile_product<128, 128, kExpertTN>(g, smem, A, B, C, g.M - t.row0, g.N - t.col0, t.rows.count);
  }
}

// ------------------------------------------------------------------------------------
// Few rows an expert: 32 x 128 or 64 x 128 tiles, four waves of 32 columns, k-tiles of 64 through a ring
// of STAGES slots, one barrier each: after the barrier of tile t the copies of tile t + STAGES - 1 go
// into the slot of tile t - 1, which every wave has read. Bound by reading the weights of the
// experts that are met: 2048 rows on 64 experts of 2048 x 2048 (32 rows a tile) 111 us, 4096 rows (64 rows
// a tile) 127, of 537 MB of weights (98 us at a copy's rate).
template <int BM>
constexpr int kSmallStages = BM == 32 ? 4 : 3;  // two workgroups a compute unit
template <int BM_, ExpertForm F>
struct SmallTile {
  static constexpr int BM = BM_, BN = 128, BK = 64, NW = 4, STAGES = kSmallStages<BM_>;
  using OpA = PpOperand<BM, BK, 16, true, NW>;
  using OpB = PpOperand<BN, BK, 16, F == kExpertNT, NW>;
  static constexpr int PT = OpA::LD + OpB::LD, SLOT = OpA::BYTES + OpB::BYTES, LDS = STAGES * SLOT;
  static_assert(OpA::REM == 0 && OpB::REM == 0, "copies split evenly");
};

template <int BM_, ExpertForm F>
__global__ __launch_bounds__(256) void expert_small(ExpertGemmArgs g) {
  using T = SmallTile<BM_, F>;
  using OpA = typename T::OpA;
  using OpB = typename T::OpB;
  constexpr int BM = T::BM, BN = T::BN, BK = T::BK, NW = T::NW, STAGES = T::STAGES, FM = BM / 16;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const RowTile t = find_tile<BM, 4>(g, lane);
  if (t.e < 0) return zero_rest<256>(g, t.past, t.past_count);
  const int row0 = t.tm * BM, col0 = t.tn * BN;
  const int mvalid = min(BM, t.rows.count - row0), nvalid = min(BN, g.N - col0);
  const int nk = k_tiles(g.K, BK), kin_last = g.K - (nk - 1) * BK;
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
  float4v acc[FM][2];
#pragma unroll
  for (int i = 0; i < FM; ++i)
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
      half8 fa[FM], fb[2];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = opa.frag(As, i, ks);
#pragma unroll
      for (int i = 0; i < 2; ++i) fb[i] = opb.frag(Bs, i, ks);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  wait_vmcnt<0>();
  __syncthreads();  // the ring is free for staging
  using ST = StagedTile<BM, 32>;
  static_assert(NW * ST::BYTES <= T::LDS, "staged tiles");
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  store_staged<ST, BM, false>(stage, lane, g.C + (int64_t)(t.rows.first + row0) * g.ldc + col0 + wave * 32, g.ldc, mvalid,
                              nvalid - wave * 32, g.vec_c);
}

// ------------------------------------------------------------------------------------
// Any alignment, stride and size: 128 x 128 tiles, four waves of 64 x 64, k-tiles of 64 through two LDS
// slots in the layout of the tile kernels (PpOperand), but filled through registers: loads of any
// address, cut by the rows' ends. Bound by their latency, of which one k-tile's products cover a part: 4096
// rows, 8 experts, 2048 x 2048: 86 us in the rows' forms and 65 in the weights' (the tile kernels 46 to 53);
// 16 rows, 8 experts of 2047 x 2047: 58 us.
template <ExpertForm F>
__global__ __launch_bounds__(256) void expert_generic(ExpertGemmArgs g) {
  constexpr int BM = 128, BK = 64;
  using OpA = PpOperand<BM, BK, 16, F != kExpertTN, 4>;
  using OpB = PpOperand<BM, BK, 16, F == kExpertNT, 4>;
  constexpr int UNITS = OpA::UNITS / 256;  // 16-byte units a thread and operand
  static_assert(OpA::UNITS == 1024 && OpB::UNITS == 1024, "units split evenly");
  __shared__ __attribute__((aligned(16))) char smem[2 * (OpA::BYTES + OpB::BYTES)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    A = g.A + (int64_t)r.first * g.lda + row0;
    B = g.B + (int64_t)r.first * g.ldb + col0;
    C = g.C + e * g.stride_c;
  } else {
    const RowTile t = find_tile<BM, 4>(g, lane);
    if (t.e < 0) return zero_rest<256>(g, t.past, t.past_count);
    row0 = t.tm * BM;
    col0 = t.tn * BM;
    mvalid = t.rows.count - row0;
    K = g.K;
    A = g.A + ((int64_t)t.rows.first + row0) * g.lda;
    B = g.B + t.e * g.stride_b + (F == kExpertNT ? (int64_t)col0 * g.ldb : col0);
    C = g.C + (int64_t)t.rows.first * g.ldc;
  }
  const int nvalid = g.N - col0;
  // Unit u of a k-tile lies at byte 16 u of the slot and holds the chunk that the swizzle puts there.
  auto fetch = [&](auto op, const _Float16* X, int64_t ld, int valid, int kt, half8 (&v)[UNITS]) __attribute__((always_inline)) {
    using Op = decltype(op);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = i * 256 + tid, line = u / Op::CPR, c = 8 * ((u % Op::CPR) ^ Op::swz(line));
      const int k = BK * kt + (Op::KMAJOR ? c : line), r = Op::KMAJOR ? line : c;
      v[i] = Op::KMAJOR ? load_half8(X + (int64_t)r * ld + k, k, r < valid ? K - k : 0)
                        : load_half8(X + (int64_t)k * ld + r, r, k < K ? valid - r : 0);
    }
  };
  auto put = [&](char* slot, const half8 (&v)[UNITS]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) *(TG_LDS half8*)(slot + (i * 256 + tid) * 16) = v[i];
  };
  OpA opa;
  OpB opb;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  opa.init_frags(wm, lane);
  opb.init_frags(wn, lane);
  float4v acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  half8 av[UNITS], bv[UNITS];
  const int nk = k_tiles(K, BK);
  if (nk > 0) {
    fetch(OpA{}, A, g.lda, mvalid, 0, av);
    fetch(OpB{}, B, g.ldb, nvalid, 0, bv);
    put(smem, av);
    put(smem + OpA::BYTES, bv);
  }
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    char* const As = smem + (kt & 1) * (OpA::BYTES + OpB::BYTES);
    char* const next = smem + (~kt & 1) * (OpA::BYTES + OpB::BYTES);
    if (kt + 1 < nk) {
      fetch(OpA{}, A, g.lda, mvalid, kt + 1, av);
      fetch(OpB{}, B, g.ldb, nvalid, kt + 1, bv);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      half8 fa[4], fb[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        fa[f] = opa.frag(As, f, ks);
        fb[f] = opb.frag(As + OpA::BYTES, f, ks);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    if (kt + 1 < nk) {
      put(next, av);
      put(next + OpA::BYTES, bv);
    }
    __syncthreads();
  }
  using ST = StagedTile<64, 64>;
  static_assert(4 * ST::BYTES <= (int)sizeof(smem), "staged tiles");
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  store_staged<ST, 64, false>(stage, lane, C + (int64_t)(row0 + wm) * g.ldc + col0 + wn, g.ldc, mvalid - wm, nvalid - wn,
                              g.vec_c);
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
hipError_t launch_small(const ExpertGemmArgs& g, unsigned grid, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  return launch(expert_small<BM, F>, 256, SmallTile<BM, F>::LDS, ready, g, grid, s, device);
}
template <ExpertForm F>
hipError_t launch_form(int cfg, const ExpertGemmArgs& g, unsigned grid, hipStream_t s, int device) {
  switch (cfg) {
    case kExpertTiles:
    case kExpert128:
    case kExpert256: {
      static std::atomic<uint64_t> ready{0};
      if constexpr (F == kExpertTN)
        return launch(expert_tiles_weights, 512, kTileLds + (int)sizeof(WeightTiles), ready, g, grid, s, device);
      else
        return launch(expert_tiles<F>, 512, kTileLds + (int)sizeof(TileFinder), ready, g, grid, s, device);
    }
    case kExpert32:
    case kExpert64:
      if constexpr (F != kExpertTN)
        return cfg == kExpert32 ? launch_small<32, F>(g, grid, s, device) : launch_small<64, F>(g, grid, s, device);
      else
        return hipErrorNotSupported;
    default:
      hipLaunchKernelGGL(expert_generic<F>, dim3(grid), dim3(256), 0, s, g);
      return hipGetLastError();
  }
}

}  // namespace

hipError_t launch_expert_gemm(int cfg, ExpertForm form, const ExpertGemmArgs& args, hipStream_t s, int device) {
  ExpertGemmArgs g = args;
  g.mode = cfg == kExpert128 ? kTilesSmall : cfg == kExpert256 ? kTilesBig : kTilesAuto;
  g.max_tiles = (uint32_t)expert_max_tiles(form, g.rows, g.experts, g.M, g.N);
  const int64_t grid = expert_gemm_groups(cfg, form, g.rows, g.experts, g.M, g.N);
  g.tiles_m = form == kExpertTN ? (int)ceil_div(g.M, 128) : 0;
  g.tiles_n = (int)ceil_div(g.N, 128);
  if (form == kExpertNT) return launch_form<kExpertNT>(cfg, g, (unsigned)grid, s, device);
  if (form == kExpertNN) return launch_form<kExpertNN>(cfg, g, (unsigned)grid, s, device);
  return launch_form<kExpertTN>(cfg, g, (unsigned)grid, s, device);
}

}  // namespace tgemm
