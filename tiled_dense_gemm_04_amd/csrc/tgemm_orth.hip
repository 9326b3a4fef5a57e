// tgemm_orth.hip -- gfx950 kernels of the Newton-Schulz orthogonalisation.
//
// X_0 = G / (|G|_F + 1e-7) (transposed if tall so that m <= n), then `steps` times
//   A = X X^T,  X <- a X + (b A + c A A) X,
// which drives every singular value of X towards one; the result is scale * X. A tall G keeps
// its orientation: A = X^T X and X <- a X + X (b A + c A A), so nothing is transposed.
//
// The products run on the binary16 MFMAs with float32 sums, and lose no more than float32
// products do:
//   * every matrix between them -- the iterate X, and off the diagonal A and the polynomial
//     P = a I + b A + c A A -- is held as two halves, hi + lo 2^-11 (22 bits);
//   * a product runs over its operands' halves three times, hi lo, lo hi, then, with those sums
//     scaled by 2^-11, hi hi. What is left out, lo lo, is 2^-22 of the terms;
//   * the diagonals, which dominate A and P once X is near orthogonal, stay in float32 and out of
//     the products: with A = diag(D) + E,
//       P_ij = b E_ij + c ((D_i + D_j) E_ij + (E E)_ij)        (i != j)
//       P_ii = a + b D_i + c (D_i^2 + (E E)_ii)
//       X'   = diag(P) X + offdiag(P) X.
//   A and E E are symmetric: only tiles on and above the diagonal are computed, each stored a
//   second time transposed.
// Relative errors of the result before its rounding to binary16 (which is 2.1e-4 of it; 5 or 6
// steps, matrices of 64 x 64 to 512 x 512, emulated in float64): 2e-7 to 9e-7 on random matrices,
// with or without strong directions, where float32 products lose 1e-6 to 3e-6; 8e-5 on rank one
// plus 1e-4 of noise, whose small directions the steps draw out of the large one's roundings
// (float32 products: 3e-4). With the high halves alone in the products (a third of their time)
// these are 1e-3 and 1.5e-2.
#include "tgemm_orth.h"
#include "tgemm_pingpong.h"

#include <atomic>

namespace tgemm {
namespace {

typedef float float4v __attribute__((ext_vector_type(4)));

constexpr float kLo = 2048.0f;  // the low half is held times 2^11: away from the subnormals
constexpr double kNormEps = 1e-7;

__device__ __forceinline__ float joined(_Float16 hi, _Float16 lo) { return (float)hi + (float)lo * (1.0f / kLo); }
__device__ __forceinline__ _Float16 low_half(float x, _Float16 hi) { return (_Float16)((x - (float)hi) * kLo); }

// Eight values of row r, columns c .. c + 7, of matrix bt as float32, zeros past the row (any
// alignment: one or two 16-byte loads, single ones at the row's end).
__device__ __forceinline__ void load_g(const OrthArgs& g, int bt, uint32_t r, uint32_t c, float (&v)[8]) {
  const int64_t at = (int64_t)bt * g.stride_g + (int64_t)r * g.ldg + c;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  if (r >= (uint32_t)g.R) return;
  if (c + 8 <= (uint32_t)g.C) {
    if (g.f32) {
      __builtin_memcpy(v, (const float*)g.G + at, 32);
    } else {
      half8 h;
      __builtin_memcpy(&h, (const _Float16*)g.G + at, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (c + e < (uint32_t)g.C) v[e] = g.f32 ? ((const float*)g.G)[at + e] : (float)((const _Float16*)g.G)[at + e];
  }
}

// Sums of squares of a matrix, g.nparts partial sums in float64 (squares of float32 values
// leave float32's range), four chunks of eight values per thread in flight. Bound by reading G:
// 16 x 512 x 2048 in float32 14.2 us (4.7 TB/s), 4096 x 4096 in binary16 13.8 us.
__global__ __launch_bounds__(256) void orth_norm(OrthArgs g) {
  __shared__ double w[4];
  const uint32_t part = blockIdx.x % g.nparts, bt = blockIdx.x / g.nparts;
  const uint32_t cpr = ((uint32_t)g.C + 7) / 8, total = cpr * (uint32_t)g.R;
  double s = 0.0;
  for (uint32_t u0 = part * 1024 + threadIdx.x; u0 < total; u0 += g.nparts * 1024) {
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = u0 + 256 * i, r = u / cpr;
      load_g(g, bt, u < total ? r : (uint32_t)g.R, (u - r * cpr) * 8, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (double)v[i][e] * (double)v[i][e];
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) g.parts[bt * kOrthParts + part] = (w[0] + w[1]) + (w[2] + w[3]);
}

// X_0 = G / (|G| + eps) as two halves, padded with zeros: two chunks of eight values per thread.
// Bound by memory, 8 bytes per value of float32 G: 16 x 512 x 2048 in 22.6 us (5.9 TB/s).
__global__ __launch_bounds__(256) void orth_start(OrthArgs g) {
  __shared__ double inv;
  const uint32_t rp = g.tall ? g.np : g.mp, cpr = (g.tall ? g.mp : g.np) / 8;
  const uint32_t total = rp * cpr, groups = (total + 511) / 512;
  const uint32_t bt = blockIdx.x / groups, u0 = (blockIdx.x - bt * groups) * 512 + threadIdx.x;
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = u0 + 256 * i, r = u / cpr;
    load_g(g, bt, u < total ? r : (uint32_t)g.R, (u - r * cpr) * 8, v[i]);
  }
  if (threadIdx.x < 64) {
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < (uint32_t)g.nparts; i += 64) s += g.parts[bt * kOrthParts + i];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
    if (threadIdx.x == 0) inv = 1.0 / (sqrt(s) + kNormEps);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = u0 + 256 * i;
    if (u >= total) continue;
    half8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = (float)((double)v[i][e] * inv);
      hi[e] = (_Float16)x;
      lo[e] = low_half(x, hi[e]);
    }
    const int64_t o = ((int64_t)bt * total + u) * 8;
    *(half8*)(g.hi[0] + o) = hi;
    *(half8*)(g.lo[0] + o) = lo;
  }
}

// ------------------------------------------------------------------------------------
// The three products of a step, one ping-pong kernel each (tgemm_pingpong.h) on BM x BM
// tiles of one matrix of the batch; what differs is the operands and the epilogue. Bound by the
// MFMAs of the three passes: 4096 x 4096: Gram 229 to 249 us and Square 241 to 258 (136 tiles on and
// above the diagonal, one per compute unit, 120 units idle; a whole 4096^3 product of the binary16
// kernels takes 106), Apply 318 to 330 (1.3 PFLOP/s). 16 x 512 x 2048: 46, 23.5 and 65 us, of which
// Apply's passes are 34 at 1.52 PFLOP/s; its epilogue moves 134 MB, 23 us at a copy's rate.
enum Product { kGram, kSquare, kApply };

struct OrthStep {
  int in, last;  // which of the two iterate buffers is read; the final step writes the result
};

template <int BM>
constexpr int kOrthKg = BM == 128 ? 2 : 1;

template <int BM>
constexpr int orth_lds_bytes() {
  // the operand ring, or the staged tiles of the epilogue (per wave, transposed with a 16-byte
  // pad per column), whichever is larger
  constexpr int ring = 4 * 2 * BM * 64 * kOrthKg<BM>, st = 8 * (BM * kOrthKg<BM> / 4) * (BM / kOrthKg<BM> + 16);
  return ring > st ? ring : st;
}

template <bool JOINED, typename A, typename B>
__device__ __forceinline__ auto& pick_sums(A& own, B& joined) {
  if constexpr (JOINED)
    return joined;
  else
    return own;
}

template <Product P, int BM, bool TALL>
__global__ __launch_bounds__(512) void orth_product(OrthArgs g, OrthStep st) {
  // Wave tiles of BM / 2 x BM / WN. Smaller tiles (KG = 2): k-tiles of 64, of which each wave
  // group takes one half on wave tiles of 64 x 64 -- a third fewer LDS reads than 64 x 32 tiles
  // over the whole of it, and LDS is what bounds them.
  constexpr int NW = 8, STAGES = 4, KG = kOrthKg<BM>, WN = 4 / KG, BK = 32 * KG;
  constexpr int WTN = BM / WN, FM = BM / 32, FN = WTN / 16;
  constexpr int WTM = BM / 2 / KG, FE = FM / KG;  // after the groups are joined
  // Gram: rows of the wide iterate, or columns of the tall one; Square: E is its own
  // transpose; Apply: P times the wide iterate (k along its rows), or the tall one times P.
  constexpr bool A_KMAJ = P != kGram || !TALL, B_KMAJ = P == kSquare || (P == kGram) != TALL;
  using OpA = PpOperand<BM, BK, 16, A_KMAJ, NW>;
  using OpB = PpOperand<BM, BK, 16, B_KMAJ, NW>;
  constexpr int A_BYTES = OpA::BYTES, B_BYTES = OpB::BYTES, PT = OpA::LD + OpB::LD;
  static_assert(OpA::REM == 0 && OpB::REM == 0, "copies split evenly");

  extern __shared__ __attribute__((aligned(16))) char smem[];
  char* const a_lds = smem;
  char* const b_lds = smem + STAGES * A_BYTES;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int rows = P == kApply && TALL ? g.np : g.mp, cols = P == kApply && !TALL ? g.np : g.mp;
  const int K = P == kGram ? g.np : g.mp;
  const int tiles_m = (rows + BM - 1) / BM, tiles_n = (cols + BM - 1) / BM;
  const int tiles = P == kApply ? tiles_m * tiles_n : tiles_n * (tiles_n + 1) / 2;
  const int64_t lid = xcd_logical_id(blockIdx.x, (int64_t)tiles * g.batch, 1);
  const int bt = (int)(lid / tiles), t = (int)(lid % tiles);
  int tm, tn;
  if (P == kApply) {
    int64_t a, b;
    panel_tile(t, tiles_m, tiles_n, 4, &a, &b);
    tm = (int)a;
    tn = (int)b;
  } else {  // tile t of the upper triangle, column by column
    tn = (int)((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (tn * (tn + 1) / 2 > t) --tn;
    while ((tn + 1) * (tn + 2) / 2 <= t) ++tn;
    tm = t - tn * (tn + 1) / 2;
  }
  const int row0 = tm * BM, col0 = tn * BM;
  const int mvalid = min(BM, rows - row0), nvalid = min(BM, cols - col0);
  const int nk = K / BK;

  const int64_t xsz = (int64_t)g.mp * g.np, esz = (int64_t)g.mp * g.mp;
  const _Float16* const hi = g.hi[st.in] + bt * xsz;
  const _Float16* const lo = g.lo[st.in] + bt * xsz;
  const _Float16* const E[2] = {g.E[0] + bt * esz, g.E[1] + bt * esz};
  float* const D = g.D + (int64_t)bt * g.mp;
  float* const DP = g.DP + (int64_t)bt * g.mp;
  const int ldx = TALL ? g.mp : g.np;  // the iterate's row length
  const _Float16* const PM[2] = {g.P[0] + bt * esz, g.P[1] + bt * esz};
  const bool a_is_x = P == kGram || (P == kApply && TALL), b_is_x = P == kGram || (P == kApply && !TALL);
  const _Float16* const Aop[2] = {a_is_x ? hi : P == kSquare ? E[0] : PM[0], a_is_x ? lo : P == kSquare ? E[1] : PM[1]};
  const _Float16* const Bop[2] = {b_is_x ? hi : P == kSquare ? E[0] : PM[0], b_is_x ? lo : P == kSquare ? E[1] : PM[1]};
  const int lda = a_is_x ? ldx : g.mp, ldb = b_is_x ? ldx : g.mp;

  OpA opa;
  OpB opb;
  opa.init_copies(Aop[0], lda, row0, mvalid, BK, wave, lane);
  opb.init_copies(Bop[0], ldb, col0, nvalid, BK, wave, lane);
  const uint32_t a_lds0 = lds_addr(a_lds) + wave * 1024, b_lds0 = lds_addr(b_lds) + wave * 1024;
  // The k-loop runs over the operands' halves three times: hi lo, lo hi, and, with the sums of
  // those scaled back, hi hi. (K is a multiple of the k-tile: every tile is whole.)
  const int64_t a_low = (const char*)Aop[1] - (const char*)Aop[0], b_low = (const char*)Bop[1] - (const char*)Bop[0];
  const char *a_next = opa.base, *b_next = opb.base + b_low;
  int ct = 0, pass = 0;  // the tile copied next
  auto copy_tile = [&](int kt, auto) __attribute__((always_inline)) {
    const int4v ra = make_rsrc(a_next, pass < 3 ? opa.rng_full : 0u), rb = make_rsrc(b_next, pass < 3 ? opb.rng_full : 0u);
    a_next += opa.step;
    b_next += opb.step;
    if (++ct == nk) {
      ct = 0;
      ++pass;
      a_next = opa.base + (pass == 1 ? a_low : 0);
      b_next = opb.base;
    }
    const int slot = kt % STAGES;
#pragma unroll
    for (int j = 0; j < OpA::LD; ++j) dma_to_lds(ra, a_lds0 + slot * A_BYTES + j * NW * 1024, opa.off[j]);
#pragma unroll
    for (int j = 0; j < OpB::LD; ++j) dma_to_lds(rb, b_lds0 + slot * B_BYTES + j * NW * 1024, opb.off[j]);
  };
  const int kg = KG == 2 ? wave >> 2 : 0, wv = wave % (2 * WN), wm = wv / WN, wn = wv % WN;
  const int lrow = lane & 15, lkg = lane >> 4;
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
  int low_left = 2 * nk;  // tiles of the passes with a low half
  auto mma_tile = [&]() __attribute__((always_inline)) {
    if (low_left-- == 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) sum[i][j] *= 1.0f / kLo;
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        sum[fm][fn] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[fn], fa[fm], sum[fm][fn], 0, 0, 0);
  };
  pingpong_schedule<STAGES, PT, PT, (A_KMAJ && B_KMAJ && BM == 256)>(wave / 4, 3 * nk, copy_tile, read_tile, mma_tile);
  __syncthreads();  // the ring is free for staging
  float4v joined_sum[KG == 2 ? FE : 1][FN];
  if constexpr (KG == 2) join_k_groups<FM, FN>(smem, sum, joined_sum, wave, lane);
  float4v(&acc)[FE][FN] = pick_sums<KG == 2>(sum, joined_sum);

  // Epilogue. The lane holds row r and columns c .. c + 3 of each 16 x 16 tile; the padded sizes
  // are multiples of 64, so a group of four lies inside the matrix or outside it.
  const int wr0 = row0 + wm * (BM / 2) + kg * WTM, wc0 = col0 + wn * WTN;
  using ST = StagedTile<WTM, WTN>;
  char* const stage = smem + wave * (orth_lds_bytes<BM>() / NW);
  static_assert(ST::BYTES <= orth_lds_bytes<BM>() / NW, "staged tile");
  const int rv = rows - wr0, cv = cols - wc0;
  // What the high halves of the sums leave, in their place (rounded again: the rounded values
  // kept from the staging would spill).
  auto take_low = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int fm = 0; fm < FE; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) {
        asm volatile("" : "+v"(acc[fm][fn]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = acc[fm][fn][e];
          acc[fm][fn][e] = (x - (float)(_Float16)x) * kLo;
        }
      }
  };

  if constexpr (P == kApply) {
    // X' = diag(P) X + offdiag(P) X. The old values of kAhead rows of tiles are in flight.
    constexpr int kAhead = FE < 3 ? FE : 3;
    half4 h[kAhead][FN], l[kAhead][FN];
    float dr[kAhead];
    auto fetch = [&](auto fm_c) __attribute__((always_inline)) {
      constexpr int fm = decltype(fm_c)::value;
      const int r = wr0 + 16 * fm + lrow, rr = min(r, rows - 1);
      dr[fm % kAhead] = TALL ? 0.0f : DP[rr];
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) {
        const int c = min(wc0 + 16 * fn + 4 * lkg, cols - 4);
        h[fm % kAhead][fn] = *(const half4*)(hi + (int64_t)rr * ldx + c);
        l[fm % kAhead][fn] = *(const half4*)(lo + (int64_t)rr * ldx + c);
      }
    };
    float4v dc[FN];
    if constexpr (TALL) {
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) dc[fn] = *(const float4v*)(DP + min(wc0 + 16 * fn + 4 * lkg, cols - 4));
    }
    static_for<kAhead>([&](auto i) __attribute__((always_inline)) { fetch(i); });
    static_for<FE>([&](auto fm_c) __attribute__((always_inline)) {
      constexpr int fm = decltype(fm_c)::value;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[fm][fn][e] += (TALL ? dc[fn][e] : dr[fm % kAhead]) * joined(h[fm % kAhead][fn][e], l[fm % kAhead][fn][e]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (fm + kAhead < FE) fetch(std::integral_constant<int, fm + kAhead>{});
    });
    if (st.last) {
#pragma unroll
      for (int fm = 0; fm < FE; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) acc[fm][fn] *= g.scale;
      ST::template stage<false>(stage, acc, lane);
      ST::wave_fence();
      _Float16* const X = g.X + bt * g.stride_x;
      const int vec = (reinterpret_cast<uintptr_t>(X) & 15) == 0 && g.ldx % 8 == 0;
      store_staged<ST, WTM>(stage, lane, X + (int64_t)wr0 * g.ldx + wc0, g.ldx, g.R - wr0, g.C - wc0, vec);
    } else {
      ST::template stage<false>(stage, acc, lane);
      ST::wave_fence();
      const int64_t o = bt * xsz + (int64_t)wr0 * ldx + wc0;
      store_staged<ST, WTM, false>(stage, lane, g.hi[st.in ^ 1] + o, ldx, rv, cv, 1);
      ST::wave_fence();
      take_low();
      ST::template stage<false>(stage, acc, lane);
      ST::wave_fence();
      store_staged<ST, WTM, false>(stage, lane, g.lo[st.in ^ 1] + o, ldx, rv, cv, 1);
    }
  } else {
    float* const dout = P == kGram ? D : DP;
    // Row fm of tiles: the diagonal, kept apart in float32, leaves the tile.
    auto split_diagonal = [&](auto fm_c) __attribute__((always_inline)) {
      constexpr int fm = decltype(fm_c)::value;
      const int r = wr0 + 16 * fm + lrow;
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) {
        const int d = r - (wc0 + 16 * fn + 4 * lkg);  // 0 .. 3: the lane holds the diagonal's value
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (d == e) {
            if (r < rows) dout[r] = acc[fm][fn][e];
            acc[fm][fn][e] = 0.0f;
          }
      }
    };
    if constexpr (P == kSquare) {
      // P from E, D and E E; the E values of kAhead rows of tiles are in flight
      constexpr int kAhead = 2;  // (three rows spill)
      half4 h[kAhead][FN], l[kAhead][FN];
      float dr[kAhead];
      float4v dc[FN];
      auto fetch = [&](auto fm_c) __attribute__((always_inline)) {
        constexpr int fm = decltype(fm_c)::value;
        const int rr = min(wr0 + 16 * fm + lrow, rows - 1);
        dr[fm % kAhead] = D[rr];
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
          const int64_t o = (int64_t)rr * g.mp + min(wc0 + 16 * fn + 4 * lkg, cols - 4);
          h[fm % kAhead][fn] = *(const half4*)(E[0] + o);
          l[fm % kAhead][fn] = *(const half4*)(E[1] + o);
        }
      };
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) dc[fn] = *(const float4v*)(D + min(wc0 + 16 * fn + 4 * lkg, cols - 4));
      static_for<kAhead>([&](auto i) __attribute__((always_inline)) { fetch(i); });
      static_for<FE>([&](auto fm_c) __attribute__((always_inline)) {
        constexpr int fm = decltype(fm_c)::value;
        __builtin_amdgcn_sched_barrier(0);
        const int r = wr0 + 16 * fm + lrow;
        const float d = dr[fm % kAhead];
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = acc[fm][fn][e], y = joined(h[fm % kAhead][fn][e], l[fm % kAhead][fn][e]);
            acc[fm][fn][e] = r == wc0 + 16 * fn + 4 * lkg + e ? g.a + g.b * d + g.c * (d * d + s)
                                                             : g.b * y + g.c * ((d + dc[fn][e]) * y + s);
          }
        split_diagonal(fm_c);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (fm + kAhead < FE) fetch(std::integral_constant<int, fm + kAhead>{});
      });
    } else {
      static_for<FE>([&](auto fm_c) __attribute__((always_inline)) { split_diagonal(fm_c); });
    }
    // One half of the tile, and off the diagonal its transpose: columns of the wave's tile become
    // rows, through LDS at WTM halves and 16 bytes a column (the pad moves neighbouring columns to
    // other banks).
    auto write = [&](_Float16* out) __attribute__((always_inline)) {
      ST::template stage<false>(stage, acc, lane);
      ST::wave_fence();
      store_staged<ST, WTM, false>(stage, lane, out + (int64_t)wr0 * g.mp + wc0, g.mp, rv, cv, 1);
      ST::wave_fence();
      if (tm == tn) return;
      constexpr int PITCH = WTM * 2 + 16;
      static_assert(WTN * PITCH <= orth_lds_bytes<BM>() / NW, "transposed tile");
#pragma unroll
      for (int fm = 0; fm < FE; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) asm volatile("" : "+v"(acc[fm][fn]));  // (rounded again, as in take_low)
#pragma unroll
      for (int fm = 0; fm < FE; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *(TG_LDS _Float16*)(stage + (16 * fn + 4 * lkg + e) * PITCH + (16 * fm + lrow) * 2) = (_Float16)acc[fm][fn][e];
      ST::wave_fence();
      constexpr int CPR = WTM / 8;
#pragma unroll
      for (int i = 0; i < WTN * CPR / 64; ++i) {
        const int u = i * 64 + lane, c = u / CPR, ch = u % CPR;
        const half8 v = *(const TG_LDS half8*)(stage + c * PITCH + ch * 16);
        if (c < cv && 8 * ch < rv) *(half8*)(out + (int64_t)(wc0 + c) * g.mp + wr0 + 8 * ch) = v;
      }
      ST::wave_fence();
    };
    _Float16* const* const out = P == kGram ? g.E : g.P;
    write(out[0] + bt * esz);
    take_low();
    write(out[1] + bt * esz);
  }
}

template <Product P, int BM, bool TALL>
hipError_t launch_product(const OrthArgs& g, OrthStep st, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  void (*const kern)(OrthArgs, OrthStep) = orth_product<P, BM, TALL>;
  constexpr int lds = orth_lds_bytes<BM>();
  const uint64_t bit = 1ull << (device & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t tm = ceil_div(g.mp, BM), tn = ceil_div(P == kApply ? g.np : g.mp, BM);
  const int64_t tiles = P == kApply ? tm * tn : tn * (tn + 1) / 2;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * g.batch)), dim3(512), lds, s, g, st);
  return hipGetLastError();
}

// 256 x 256 tiles where they fill half of the 256 compute units, else 128 x 128.
template <Product P>
hipError_t launch_any(const OrthArgs& g, OrthStep st, hipStream_t s, int device) {
  const int64_t tm = ceil_div(g.mp, 256), tn = ceil_div(P == kApply ? g.np : g.mp, 256);
  const bool big = (P == kApply ? tm * tn : tn * (tn + 1) / 2) * g.batch >= 128;
  if (g.tall) return big ? launch_product<P, 256, true>(g, st, s, device) : launch_product<P, 128, true>(g, st, s, device);
  return big ? launch_product<P, 256, false>(g, st, s, device) : launch_product<P, 128, false>(g, st, s, device);
}

}  // namespace

hipError_t launch_orthogonalize(const OrthArgs& g, int steps, hipStream_t s, int device) {
  hipLaunchKernelGGL(orth_norm, dim3((unsigned)g.batch * g.nparts), dim3(256), 0, s, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t groups = ceil_div((int64_t)g.mp * g.np / 8, 512);
  hipLaunchKernelGGL(orth_start, dim3((unsigned)(groups * g.batch)), dim3(256), 0, s, g);
  e = hipGetLastError();
  for (int i = 0; i < steps && e == hipSuccess; ++i) {
    const OrthStep st{i & 1, i == steps - 1};
    e = launch_any<kGram>(g, st, s, device);
    if (e == hipSuccess) e = launch_any<kSquare>(g, st, s, device);
    if (e == hipSuccess) e = launch_any<kApply>(g, st, s, device);
  }
  return e;
}

}  // namespace tgemm
