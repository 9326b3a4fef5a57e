// tgemm_mx.hip -- gfx950 kernels of the MXFP4 operators: the quantiser and its inverse, the
// product of two MXFP4 matrices, and the product of a binary16 matrix with an MXFP4 weight.
//
// An MXFP4 matrix holds E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) in blocks of 32
// along k, each with one E8M0 scale 2^(s - 127). Rows hold whole blocks (16 bytes each), zero
// codes past K:
//   quantiser:  s = floor(log2 max|x|) - 2 + 127, code = E2M1(x 2^(127 - s)), to nearest even,
//               saturated at 6 (7 < x 2^.. < 8 rounds past the grid);
//   products:   C[i,j] = ReLU?( sum_kb 2^(sa + sb - 254) sum_{k in kb} a[i,k] b[j,k] ), or with
//               binary16 A and the weight decoded to binary16, sum_k a[i,k] half(2^(sb - 127)
//               b[j,k]), both summed in float32 and rounded to binary16 once.
#include "tgemm_mx.h"
#include "tgemm_pingpong.h"

#include <atomic>

namespace tgemm {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
typedef unsigned int uint2v __attribute__((ext_vector_type(2)));
typedef unsigned int uint4v __attribute__((ext_vector_type(4)));

// Loads and stores of any alignment (gfx950 serves them; the compiler emits one wide access).
template <typename V>
__device__ __forceinline__ V load_any(const void* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}
template <typename V>
__device__ __forceinline__ void store_any(void* p, const V& v) {
  __builtin_memcpy(p, &v, sizeof(V));
}

// 2^(s - 127) as float32; s = 0 is a subnormal, 255 a NaN.
__device__ __forceinline__ float scale_f32(uint32_t s) {
  return __uint_as_float(s == 255 ? 0x7FC00000u : s == 0 ? 0x00400000u : s << 23);
}

// Lane permutations inside groups of four lanes.
__device__ __forceinline__ uint32_t quad_xor1(uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true); }
__device__ __forceinline__ uint32_t quad_xor2(uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true); }

// Rotation by N lanes inside rows of 16.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x120 + N, 0xF, 0xF, true); }

// Magnitudes of binary16 values order like their bit patterns, infinities and NaN at the top.
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  const ushort2v x = __builtin_bit_cast(ushort2v, a), y = __builtin_bit_cast(ushort2v, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}
constexpr uint32_t kAbs2 = 0x7FFF7FFFu;

// The scale byte of a block whose largest magnitude has binary16 bits h: the exponent of that
// magnitude minus 2 (E2M1's largest exponent), 127 (a scale of one) for a block of zeros, 255
// where the block holds an infinity or a NaN. Every nonzero magnitude (at least 2^-24) is a
// normal float32, so its exponent field is the logarithm.
__device__ __forceinline__ uint32_t scale_byte(uint32_t h) {
  const float f = (float)__builtin_bit_cast(_Float16, (unsigned short)h);
  const uint32_t e = (__float_as_uint(f) >> 23) - 2;
  return h == 0 ? 127u : h >= 0x7C00u ? 255u : e;
}

// Two binary16 values to two E2M1 codes in byte B of a word: x / scale to nearest even,
// saturated at 6 (gfx950's conversion; checked code by code against the definition).
template <int B>
__device__ __forceinline__ uint32_t fp4_pack(uint32_t old, uint32_t x, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(half2v, x), scale, B);
}
// Eight binary16 values (four words) to eight codes; a block with scale byte 255 gets zeros.
__device__ __forceinline__ uint32_t fp4_pack8(const uint4v& x, uint32_t sb) {
  const float s = __uint_as_float(sb << 23);
  uint32_t w = 0;
  w = fp4_pack<0>(w, x[0], s);
  w = fp4_pack<1>(w, x[1], s);
  w = fp4_pack<2>(w, x[2], s);
  w = fp4_pack<3>(w, x[3], s);
  return sb == 255 ? 0u : w;
}

// Eight consecutive binary16 values from p, those at or past `n` zero.
__device__ __forceinline__ uint4v load8(const _Float16* p, int n) {
  uint4v v = {0, 0, 0, 0};
  if (n >= 8) {
    v = load_any<uint4v>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) v[e / 2] |= (uint32_t)__builtin_bit_cast(unsigned short, p[e]) << (16 * (e % 2));
  }
  return v;
}

// ------------------------------------------------------------------------------------
// Quantiser along the rows. Four lanes per block, eight values (16 bytes) each, NB blocks per
// group of lanes with all loads issued first; block b of the matrix is block b % KB of row
// b / KB, so consecutive groups of lanes read consecutive memory. Bound by memory: 2 bytes
// read and 17/32 written per value; 16384 x 4096 takes 30.8 us, 5.5 TB/s, the rate of a plain
// copy.
template <int NB>
__global__ __launch_bounds__(256) void quant_mxfp4_rows(MxQuantArgs q) {
  const uint32_t KB = (uint32_t)((q.K - 1) / kMxBlock + 1);
  const uint64_t nblk = (uint64_t)q.R * KB;
  const int sub = threadIdx.x & 3;
  const uint64_t first = (uint64_t)blockIdx.x * (64 * NB) + (threadIdx.x >> 2);
  uint4v x[NB];
  uint32_t row[NB], kb[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const uint64_t b = first + 64 * i;  // the host keeps the number of blocks below 2^32
    row[i] = (uint32_t)b / KB;
    kb[i] = (uint32_t)b - row[i] * KB;
    x[i] = (uint4v){0, 0, 0, 0};
    if (b < nblk) x[i] = load8(q.X + (int64_t)row[i] * q.ldx + kb[i] * kMxBlock + 8 * sub, q.K - (int)(kb[i] * kMxBlock + 8 * sub));
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    uint32_t m = pk_max(pk_max(x[i][0] & kAbs2, x[i][1] & kAbs2), pk_max(x[i][2] & kAbs2, x[i][3] & kAbs2));
    m = pk_max(m, quad_xor1(m));
    m = pk_max(m, quad_xor2(m));
    const uint32_t sb = scale_byte(m >> 16 > (m & 0xFFFF) ? m >> 16 : m & 0xFFFF);
    if (first + 64 * i >= nblk) continue;
    store_any(q.Q + (int64_t)row[i] * q.ldq + kb[i] * kMxBlockBytes + 4 * sub, fp4_pack8(x[i], sb));
    if (sub == 0) q.S[(int64_t)row[i] * q.lds + kb[i]] = (uint8_t)sb;
  }
}

// ------------------------------------------------------------------------------------
// Quantiser along the columns (blocks of 32 rows, codes of X^T), and with ROWS along the rows
// in the same pass over X. A workgroup takes 256 rows x 128 columns. Wave w takes row blocks
// w and w + 4; a lane holds 8 rows x 8 columns of a block (lane % 16: columns, lane / 16:
// rows), so a row of the tile is one 256-byte load, a column's maximum is one over the lane's
// rows and two lane swaps, and a row block's one over four neighbouring lanes. The codes of
// X^T cross the workgroup through LDS ([128 columns][8 blocks of 16 bytes], block j of column
// c at place j ^ (c / 8) % 8, which spreads the sixteen columns groups written at once over
// the banks) and leave as 128 contiguous bytes per column. Bound by memory and by the strided
// rows and columns it is reached through: 16384 x 4096 along the columns 36.5 us (4.7 TB/s), along
// both axes 50 to 52 us (4.0 TB/s; two passes would read X twice and take 67). The 13 us between them
// are the rows' codes and scales, 36 MB in pieces of 64 (half a line, a tile being 128 columns wide)
// and 4 bytes: 6 us at a copy's rate.
template <bool ROWS>
__global__ __launch_bounds__(256) void quant_mxfp4_cols(MxQuantArgs q) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[128 * 128];
  __shared__ __attribute__((aligned(8))) uint8_t scales[128 * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cg = lane & 15, sub = lane >> 4;
  const uint32_t tiles_c = (uint32_t)((q.K + 127) / 128);
  const int r0 = (int)(blockIdx.x / tiles_c) * 256, c0 = (int)(blockIdx.x % tiles_c) * 128;
  const int RB = (q.R - 1) / kMxBlock + 1, rb0 = r0 / kMxBlock;
  const int col = c0 + 8 * cg;
  // Tiles inside the matrix are loaded without checks (4096 x 4096 along both axes: 14.0 -> 13.3
  // us). Columns alone: both row blocks' loads come first (2048 x 1024: 5.2 -> 4.5 us, 16384 x
  // 4096: 37.4 -> 36.5); beside the rows' work that measured slower (50 -> 52 us).
  constexpr int AHEAD = ROWS ? 1 : 2;
  uint4v xs[AHEAD][8];
  auto load = [&](int h, bool checked) __attribute__((always_inline)) {
    const int row = r0 + (wave + 4 * h) * kMxBlock + 8 * sub;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint4v& v = xs[h % AHEAD][r];
      const _Float16* const p = q.X + (int64_t)(row + r) * q.ldx + col;
      if (!checked) {
        v = load_any<uint4v>(p);
      } else {
        v = (uint4v){0, 0, 0, 0};
        if (row + r < q.R && col < q.K) v = load8(p, q.K - col);
      }
    }
  };
  const bool whole = r0 + 256 <= q.R && c0 + 128 <= q.K;
  auto load_range = [&](int lo, int hi) __attribute__((always_inline)) {
    if (whole) {
      for (int h = lo; h < hi; ++h) load(h, false);
    } else {
      for (int h = lo; h < hi; ++h) load(h, true);
    }
  };
  if (!ROWS) load_range(0, 2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = wave + 4 * h;
    const int row = r0 + j * kMxBlock + 8 * sub;
    if (ROWS) load_range(h, h + 1);
    uint4v(&x)[8] = xs[h % AHEAD];
    if (ROWS) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        uint32_t m = pk_max(pk_max(x[r][0] & kAbs2, x[r][1] & kAbs2), pk_max(x[r][2] & kAbs2, x[r][3] & kAbs2));
        m = pk_max(m, quad_xor1(m));
        m = pk_max(m, quad_xor2(m));
        const uint32_t sb = scale_byte(m >> 16 > (m & 0xFFFF) ? m >> 16 : m & 0xFFFF);
        // a block that starts inside the row is written whole, zero codes past K
        const bool in = row + r < q.R && (col & ~(kMxBlock - 1)) < q.K;
        if (in) store_any(q.Q + (int64_t)(row + r) * q.ldq + col / 2, fp4_pack8(x[r], sb));
        // the row's four scale bytes leave as one word
        uint32_t s4 = sb << (8 * (cg >> 2));
        s4 |= row_ror<4>(s4);
        s4 |= row_ror<8>(s4);
        uint8_t* const sp = q.S + (int64_t)(row + r) * q.lds + c0 / kMxBlock;
        if (c0 + 96 < q.K) {
          if (cg == 0 && in) store_any(sp, s4);
        } else if ((cg & 3) == 0 && in) {
          sp[cg >> 2] = (uint8_t)sb;
        }
      }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // columns 2p and 2p + 1
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) m = pk_max(m, x[r][p] & kAbs2);
      m = pk_max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = pk_max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      const uint32_t sb0 = scale_byte(m & 0xFFFF), sb1 = scale_byte(m >> 16);
      uint4v lo, hi;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        lo[r] = __builtin_amdgcn_perm(x[2 * r + 1][p], x[2 * r][p], 0x05040100);
        hi[r] = __builtin_amdgcn_perm(x[2 * r + 1][p], x[2 * r][p], 0x07060302);
      }
      const int at = 8 * cg + 2 * p, place = ((j ^ (cg & 7)) << 4) + 4 * sub;
      *(TG_LDS uint32_t*)(codes + at * 128 + place) = fp4_pack8(lo, sb0);
      *(TG_LDS uint32_t*)(codes + (at + 1) * 128 + place) = fp4_pack8(hi, sb1);
      if (sub == 0) {
        *(TG_LDS uint8_t*)(scales + at * 8 + j) = (uint8_t)sb0;
        *(TG_LDS uint8_t*)(scales + (at + 1) * 8 + j) = (uint8_t)sb1;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = i * 256 + threadIdx.x, c = u >> 3, j = u & 7;
    const uint4v v = *(const TG_LDS uint4v*)(codes + c * 128 + ((j ^ ((c >> 3) & 7)) << 4));
    if (c0 + c < q.K && rb0 + j < RB) {
      store_any(q.QT + (int64_t)(c0 + c) * q.ldqt + (int64_t)(rb0 + j) * kMxBlockBytes, v);
      if (rb0 + 8 > RB) q.ST[(int64_t)(c0 + c) * q.ldst + rb0 + j] = *(const TG_LDS uint8_t*)(scales + c * 8 + j);
    }
  }
  if (rb0 + 8 <= RB && threadIdx.x < 128 && c0 + (int)threadIdx.x < q.K)
    store_any(q.ST + (int64_t)(c0 + threadIdx.x) * q.ldst + rb0, *(const TG_LDS uint2v*)(scales + threadIdx.x * 8));
}

// ------------------------------------------------------------------------------------
// Codes and scales to binary16 values, each rounded to nearest even (only scales outside
// 2^-23 .. 2^13 make values that binary16 does not hold; those past its range become
// infinite, a scale byte of 255 gives NaN). Four lanes per block, eight values (16 bytes
// written) each, NB blocks per group of lanes. Bound by memory: 16384 x 4096 in 31 to 35 us
// (4.9 to 5.5 TB/s).
__device__ __forceinline__ half8 decode8(uint32_t w, uint32_t sb) {
  const float s = scale_f32(sb);
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1);
  const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3);
  return (half8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int NB>
__global__ __launch_bounds__(256) void dequant_mxfp4_rows(MxDequantArgs q) {
  const uint32_t KB = (uint32_t)((q.K - 1) / kMxBlock + 1);
  const uint64_t nblk = (uint64_t)q.R * KB;
  const int sub = threadIdx.x & 3;
  const uint64_t first = (uint64_t)blockIdx.x * (64 * NB) + (threadIdx.x >> 2);
  uint32_t w[NB], sb[NB], row[NB], kb[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const uint64_t b = first + 64 * i;
    row[i] = (uint32_t)b / KB;
    kb[i] = (uint32_t)b - row[i] * KB;
    if (b < nblk) {
      w[i] = load_any<uint32_t>(q.Q + (int64_t)row[i] * q.ldq + kb[i] * kMxBlockBytes + 4 * sub);
      sb[i] = q.S[(int64_t)row[i] * q.lds + kb[i]];
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (first + 64 * i >= nblk) continue;
    const int k = (int)(kb[i] * kMxBlock) + 8 * sub;
    _Float16* const p = q.X + (int64_t)row[i] * q.ldx + k;
    const half8 v = decode8(w[i], sb[i]);
    if (k + 8 <= q.K) {
      store_any(p, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < q.K) p[e] = v[e];
    }
  }
}

// ------------------------------------------------------------------------------------
// Products of two MXFP4 matrices. One v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by
// 128 x 16 codes and applies both operands' block scales itself: lane l's 16 bytes of an operand
// are one whole block (row l % 16) and its scale byte sits in a register beside it, so nothing
// is folded outside the MFMA. k-tiles are 256 codes, 128 bytes a row: operand copies,
// range-checked edges and swizzle are the binary16 kernels' (PpOperand on code rows seen as
// halves), and whole 128-byte lines move fastest (copies alone reach 118 GB/s per compute unit
// in long runs, 70 in 64-byte pieces). Scales come in groups of 16 blocks (two k-tiles), 16 bytes
// a row and one 16-byte copy per row. In the last group bytes past KB are whatever the padding
// holds; they meet zero codes (out-of-range copies) and are replaced or cleared.
// Requirements (host): A, B, SA, SB 16-byte aligned, their row strides multiples of 16.
//
// Small output grids: the two-group ping-pong (tgemm_pingpong.h). Each group takes half of every
// k-tile on wave tiles of 64 x 64 (128 x 128 tiles; a third fewer LDS reads than 64 x 32 tiles over
// the whole of it) or 64 x 32 (64 x 128 tiles), and the groups' sums are joined at the end. 128 x
// 128 tiles have room for four slots of 32 KB, 64 x 128 ones for six of 24 KB on twice the compute
// units. 512 x 4096 x 4096: 11.6 to 13 us on 64 x 128 tiles (14.6 on 128 x 128); 2048 x 2048 x 4096:
// 15.4 us on 128 x 128 (22.9 on 64 x 128), 2.2 PFLOP/s. By K (256 x 4096: 6.3 us at 1001, 11.0 at
// 4095) a round of 64 x 128 tiles is 4.7 us (launch, first copies, join and stores) and 0.39 a k-tile,
// whose copies at 118 GB/s are 0.2 and whose MFMAs 0.16: they do not overlap as they should, which is open.
template <int BM, int STAGES, int PANEL>
__global__ __launch_bounds__(512) void gemm_mxfp4_small(MxGemmArgs g) {
  constexpr int BN = 128, NW = 8, WN = BM == 128 ? 2 : 4, WTN = BN / WN, FM = 4, FN = WTN / 16;
  using OpA = PpOperand<BM, 64, 16, true, NW>;
  using OpB = PpOperand<BN, 64, 16, true, NW>;
  constexpr int A_SLOT = OpA::BYTES, B_SLOT = OpB::BYTES;
  constexpr int TB = 8, GROUP = 2;  // blocks per row of a k-tile, k-tiles per scale group
  // Group 1 copies scale group s with its first k-tile 2 s in iteration 2 s - STAGES + 1, when
  // that k-tile may still be read: the slot's former group s - 4 ended with k-tile 2 s - 7.
  constexpr int SLOTS = 4, SG_BYTES = (BM + BN) * 16, SC_A = BM / 64;
  static_assert(OpA::REM == 0 && OpB::REM == 0 && STAGES <= 7 && SC_A + BN / 64 <= 4, "copies");

  extern __shared__ __attribute__((aligned(16))) char smem[];
  char* const a_lds = smem;
  char* const b_lds = smem + STAGES * A_SLOT;
  char* const s_lds = b_lds + STAGES * B_SLOT;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2;
  int64_t tm, tn;
  tile_of(blockIdx.x, g.tiles_m, g.tiles_n, PANEL, 1, &tm, &tn);
  const int row0 = (int)tm * BM, col0 = (int)tn * BN;
  const int mvalid = min(BM, g.M - row0), nvalid = min(BN, g.N - col0);
  const int nk = (g.KB + TB - 1) / TB;
  const int kin_last = (g.KB - (nk - 1) * TB) * (kMxBlockBytes / 2);  // in halves

  OpA opa;
  OpB opb;
  opa.init_copies((const _Float16*)g.A, g.lda / 2, row0, mvalid, kin_last, wave, lane);
  opb.init_copies((const _Float16*)g.B, g.ldb / 2, col0, nvalid, kin_last, wave, lane);
  const uint32_t a_lds0 = lds_addr(a_lds) + wave * 1024, b_lds0 = lds_addr(b_lds) + wave * 1024;
  // The scale copies (64 rows of A or B each) are group 1's, at most one per wave.
  const int part = wave & 3;
  const bool s_is_a = part < SC_A;
  const int s_row = (s_is_a ? part : part - SC_A) * 64;
  const int64_t s_ld = s_is_a ? g.ldsa : g.ldsb;
  const uint8_t* const s_base = s_is_a ? g.SA + (int64_t)(row0 + s_row) * s_ld : g.SB + (int64_t)(col0 + s_row) * s_ld;
  const uint32_t s_off = lane < (s_is_a ? mvalid : nvalid) - s_row ? (uint32_t)lane * (uint32_t)s_ld : kOob;
  const uint32_t s_dst = lds_addr(s_lds) + part * 1024;
  TileStream ta, tb;
  ta.init(opa, nk);
  tb.init(opb, nk);
  int to = 0;  // the slot copied to next
  auto copy_tile = [&](int t, auto group) __attribute__((always_inline)) {
    if (decltype(group)::value == 1 && t % GROUP == 0 && t < nk && part < SC_A + BN / 64)
      dma_to_lds(make_rsrc(s_base + (int64_t)(t / GROUP) * 16, kMaxRange), s_dst + (t / GROUP % SLOTS) * SG_BYTES, s_off);
    const bool last = ta.at_last();
    const int4v ra = ta.next(), rb = tb.next();
    const int slot = to;
    to = to == STAGES - 1 ? 0 : to + 1;
#pragma unroll
    for (int j = 0; j < OpA::LD; ++j) dma_to_lds(ra, a_lds0 + slot * A_SLOT + j * NW * 1024, last ? opa.off_last[j] : opa.off[j]);
#pragma unroll
    for (int j = 0; j < OpB::LD; ++j) dma_to_lds(rb, b_lds0 + slot * B_SLOT + j * NW * 1024, last ? opb.off_last[j] : opb.off[j]);
  };

  const int wm = part / WN, wn = part % WN, lrow = lane & 15, lblk = lane >> 4;
  opa.init_frags(wm * 64, lane);
  opb.init_frags(wn * WTN, lane);
  const char* const sa_lds = s_lds + (wm * 64 + lrow) * 16;
  const char* const sb_lds = s_lds + (BM + wn * WTN + lrow) * 16;
  half8 fa[FM], fb[FN];
  int sa[FM], sb[FN];
  int from = 0;  // the slot read next (tiles are read in order, each once)
  auto read_tile = [&](int t) __attribute__((always_inline)) {
    const char* const As = a_lds + from * A_SLOT;
    const char* const Bs = b_lds + from * B_SLOT;
    from = from == STAGES - 1 ? 0 : from + 1;
    // (a lane whose block lies past KB takes the last block's scale)
    const int off = (t / GROUP % SLOTS) * SG_BYTES + TB * (t % GROUP) + max(min(4 * grp + lblk, g.KB - 1 - TB * t), 0);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
      fb[fn] = opb.frag(Bs, fn, grp);
      sb[fn] = *(const TG_LDS uint8_t*)(sb_lds + off + fn * 256);
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      fa[fm] = opa.frag(As, fm, grp);
      sa[fm] = *(const TG_LDS uint8_t*)(sa_lds + off + fm * 256);
    }
  };
  float4v sum[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sum[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  auto wide = [](const half8& h) {
    const int4v v = __builtin_bit_cast(int4v, h);
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
  };
  // Operands go in as (B fragment, A fragment), so a lane holds four consecutive columns.
  auto mma_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        sum[fm][fn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(fb[fn]), wide(fa[fm]), sum[fm][fn], 4, 4, 0, sb[fn], 0, sa[fm]);
  };
  pingpong_schedule<STAGES, OpA::LD + OpB::LD, OpA::LD + OpB::LD, false>(grp, nk, copy_tile, read_tile, mma_tile);

  __syncthreads();
  float4v acc[FM / 2][FN];
  join_k_groups<FM, FN>(smem, sum, acc, wave, lane);
  using ST = StagedTile<32, WTN>;
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu != 0)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  const int r0 = wm * 64 + grp * 32, c0 = wn * WTN;
  store_staged<ST, 32>(stage, lane, g.C + (int64_t)(row0 + r0) * g.ldc + col0 + c0, g.ldc, mvalid - r0, nvalid - c0, g.vec_c);
}

template <int BM, int STAGES>
constexpr int kMxSmallLds = STAGES * (BM + 128) * 128 + 4 * (BM + 128) * 16;

// ------------------------------------------------------------------------------------
// 256 x 256 tiles: two slots of k-tiles. A wave reads all fragments of a k-tile (96 registers)
// and runs its 64 MFMAs from them, so a slot is free again as soon as both groups have read it
// (four slots of 128 codes and the binary16 kernel's schedule: 8192^3 in 285 us against 260).
// Interval kt (between barriers kt - 1 and kt; tile t in slot t % 2):
//   group 0: reads tile kt; copies A's tile kt + 1; MFMAs of tile kt; waits for the copies;
//   group 1: copies B's tile kt + 1; MFMAs of tile kt - 1; reads tile kt; waits likewise.
// Tile kt + 1 goes to the slot of tile kt - 1, which both groups read before barrier kt - 1, and
// is complete for everyone after barrier kt.
// Scales: 16 blocks (two k-tiles) a row per 16-byte copy, three slots; tile t brings A's
// (t even) or B's (t odd) next group t / 2 + 1, whose slot held group t / 2 - 2. A lane's MFMA
// ks takes block 2 (l / 16) + ks of the k-tile on both sides, so its two scales of a row are
// neighbouring bytes: one 2-byte read, the MFMA picks the byte. Blocks past KB: zero codes, and
// the scale bytes (whatever the padding holds) are cleared.
// 8192^3 in 252 us (4.4 PFLOP/s). Its MFMAs alone, from registers, take 169 us for 8192^3 (power
// holds the clock at 1.74 GHz), with the loop's barriers 182, the copies and reads alone 150: what
// bounds it is the matrix pipe's power and the part of the reads that the other group's MFMAs do
// not cover. 4096^3 in 37 to 38: one round of tiles, whose 16 intervals take 31 at 8192^3's pace; its
// first copies and its epilogue have nothing to overlap with.
template <int PANEL>
__global__ __launch_bounds__(512) void gemm_mxfp4_pp256(MxGemmArgs g) {
  constexpr int BM = 256, BN = 256, WM = 2, WN = 4, NC = 4, WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
  using Op = PpOperand<256, 64, 16, true, NC>;  // both operands; the copies of four waves
  constexpr int SLOT = Op::BYTES, LD = Op::LD, TB = 8, SG_BYTES = (BM + BN) * 16;
  static_assert(LD == 8 && Op::CPR == 8, "copies");
  extern __shared__ __attribute__((aligned(16))) char smem[];
  char* const a_lds = smem;
  char* const b_lds = smem + 2 * SLOT;
  char* const s_lds = b_lds + 2 * SLOT;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave / NC, cw = wave % NC;
  int64_t tm, tn;
  tile_of(blockIdx.x, g.tiles_m, g.tiles_n, PANEL, 1, &tm, &tn);
  const int row0 = (int)tm * BM, col0 = (int)tn * BN;
  const int mvalid = min(BM, g.M - row0), nvalid = min(BN, g.N - col0);
  const int nk = (g.KB + TB - 1) / TB;
  const int kin_last = (g.KB - (nk - 1) * TB) * (kMxBlockBytes / 2);  // in halves

  Op opa, opb;
  opa.init_copies((const _Float16*)g.A, g.lda / 2, row0, mvalid, kin_last, cw, lane);
  opb.init_copies((const _Float16*)g.B, g.ldb / 2, col0, nvalid, kin_last, cw, lane);
  // Copy j of a thread lies RSTEP rows after copy 0, a multiple of the swizzle period, so its
  // offset is copy 0's plus j RSTEP rows; an out-of-range offset stays out of range and below
  // 2^32 (row strides are at most 2^23 bytes). Two registers per operand instead of 2 LD.
  constexpr int RSTEP = NC * 64 / Op::CPR;
  static_assert(RSTEP % 16 == 0 && (LD - 1) * RSTEP < 256, "copy rows");
  const uint32_t a_rstep = (uint32_t)RSTEP * (uint32_t)g.lda, b_rstep = (uint32_t)RSTEP * (uint32_t)g.ldb;
  const uint32_t a_off = opa.off[0], a_off_last = opa.off_last[0], b_off = opb.off[0], b_off_last = opb.off_last[0];
  const uint32_t a_dst = lds_addr(a_lds) + cw * 1024, b_dst = lds_addr(b_lds) + cw * 1024;
  TileStream ta, tb;
  ta.init(opa, nk);
  tb.init(opb, nk);
  auto copy_a = [&](int t) __attribute__((always_inline)) {
    const uint32_t o = ta.at_last() ? a_off_last : a_off;
    const int4v r = ta.next();
    const uint32_t d = a_dst + (t & 1) * SLOT;
#pragma unroll
    for (int j = 0; j < LD; ++j) dma_to_lds(r, d + j * NC * 1024, o + j * a_rstep);
  };
  auto copy_b = [&](int t) __attribute__((always_inline)) {
    const uint32_t o = tb.at_last() ? b_off_last : b_off;
    const int4v r = tb.next();
    const uint32_t d = b_dst + (t & 1) * SLOT;
#pragma unroll
    for (int j = 0; j < LD; ++j) dma_to_lds(r, d + j * NC * 1024, o + j * b_rstep);
  };
  // Scale group sg of A's (is_a) or B's rows 64 cw .. + 63.
  auto copy_scales = [&](int sg, bool is_a) __attribute__((always_inline)) {
    const int64_t ld = is_a ? g.ldsa : g.ldsb;
    const uint8_t* const base = is_a ? g.SA + (int64_t)(row0 + cw * 64) * ld : g.SB + (int64_t)(col0 + cw * 64) * ld;
    const int left = (is_a ? mvalid : nvalid) - cw * 64;
    dma_to_lds(make_rsrc(base + (int64_t)sg * 16, 2 * sg < nk ? kMaxRange : 0u),
               lds_addr(s_lds) + (sg % 3) * SG_BYTES + (is_a ? 0 : BM * 16) + cw * 1024,
               lane < left ? (uint32_t)lane * (uint32_t)ld : kOob);
  };

  const int wm = wave / WN, wn = wave % WN, lrow = lane & 15, lblk = lane >> 4;
  // Fragment f, substep ks: chunk 2 lblk + ks of row 16 f + lrow.
  const int sw = Op::swz(lrow);
  const char* const a_rd[2] = {a_lds + (wm * WTM + lrow) * 128 + (((2 * lblk) ^ sw) << 4),
                               a_lds + (wm * WTM + lrow) * 128 + (((2 * lblk + 1) ^ sw) << 4)};
  const char* const b_rd[2] = {b_lds + (wn * WTN + lrow) * 128 + (((2 * lblk) ^ sw) << 4),
                               b_lds + (wn * WTN + lrow) * 128 + (((2 * lblk + 1) ^ sw) << 4)};
  const char* const sa_rd = s_lds + (wm * WTM + lrow) * 16 + 2 * lblk;
  const char* const sb_rd = s_lds + (BM + wn * WTN + lrow) * 16 + 2 * lblk;
  int4v fa[2][FM], fb[2][FN];
  uint32_t sa[FM], sb[FN];
  auto read_tile = [&](int t) __attribute__((always_inline)) {
    const int slot = (t & 1) * SLOT, so = (t / 2 % 3) * SG_BYTES + (t & 1) * 8;
    const int left = g.KB - TB * t - 2 * lblk;  // blocks of this lane inside the matrix
    const uint32_t mask = left >= 2 ? 0xFFFFu : left == 1 ? 0xFFu : 0u;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) sb[fn] = *(const TG_LDS uint16_t*)(sb_rd + so + fn * 256) & mask;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) sa[fm] = *(const TG_LDS uint16_t*)(sa_rd + so + fm * 256) & mask;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) fb[ks][fn] = *(const TG_LDS int4v*)(b_rd[ks] + slot + fn * 2048);
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) fa[ks][fm] = *(const TG_LDS int4v*)(a_rd[ks] + slot + fm * 2048);
    }
  };
  float4v acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  auto wide = [](const int4v& v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); };
  auto mma_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(fb[0][fn]), wide(fa[0][fm]), acc[fm][fn], 4, 4, 0, sb[fn], 0, sa[fm]);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(fb[1][fn]), wide(fa[1][fm]), acc[fm][fn], 4, 4, 1, sb[fn], 1, sa[fm]);
  };

  if (grp == 0) {
    copy_scales(0, true);
    copy_scales(0, false);
    copy_scales(1, true);
    copy_a(0);
  } else {
    copy_b(0);
  }
  wait_vmcnt<0>();
  lds_barrier();
  // sched_barrier(0) pins every phase: MFMAs only touch registers, so s_barrier does not order
  // them.
  if (grp == 0) {
    for (int kt = 0; kt < nk; ++kt) {
      __builtin_amdgcn_sched_barrier(0);
      read_tile(kt);
      copy_a(kt + 1);
      copy_scales((kt + 1) / 2 + 1, ((kt + 1) & 1) == 0);
      __builtin_amdgcn_sched_barrier(0);
      mma_tile();
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<0>();
      lds_barrier();  // (barrier kt)
    }
  } else {
    copy_b(1);  // in interval 0
    for (int kt = 0; kt < nk; ++kt) {
      __builtin_amdgcn_sched_barrier(0);
      read_tile(kt);
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<0>();
      lds_barrier();  // (barrier kt)
      __builtin_amdgcn_sched_barrier(0);
      copy_b(kt + 2);  // in interval kt + 1
      __builtin_amdgcn_sched_barrier(0);
      mma_tile();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_vmcnt<0>();

  using ST = StagedTile<WTM, WTN>;
  static_assert(8 * ST::BYTES <= 4 * SLOT, "staged tile fits in the ring");
  __syncthreads();
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu != 0)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  store_staged<ST, WTM>(stage, lane, g.C + (int64_t)(row0 + wm * WTM) * g.ldc + col0 + wn * WTN, g.ldc,
                        mvalid - wm * WTM, nvalid - wn * WTN, g.vec_c);
}

constexpr int kMx256Lds = 4 * 256 * 128 + 3 * 512 * 16;

// ------------------------------------------------------------------------------------
// Product of binary16 A with an MXFP4 weight, ping-pong kernel on k-tiles of 32 (one block):
// A's tile as in the binary16 kernel (64-byte rows), B's 16 bytes a row. Lane l of a 16 x 16
// x 32 MFMA needs k 8 (l / 16) .. + 7 of weight row l % 16: one 4-byte LDS read (16 rows of
// 16 bytes: every bank once) and four conversions with the block's scale, done in the phase
// in which the other group's MFMAs keep the matrix pipe busy. Scales come 16 bytes a row, which
// covers 16 k-tiles, in two slots. 4096^3 in 103 to 110 us on 256 x 256 tiles (8192^3: 798 us,
// 1.38 PFLOP/s, the rate of the binary16 kernels, which MFMA issue and power bound). 512 x 4096 x
// 4096 takes 41.5 us on 128 x 128 tiles: 128 workgroups for 256 compute units, each running 128
// k-tiles at 0.29 us (K = 1001: 12.7 us). What a k-tile waits for is open; k-tiles of 64 (A's rows in 128-byte pieces
// instead of 64) measured the same, so it is not the size of the copies' pieces.
// Requirements (host): A, B, SB 16-byte aligned, lda and K multiples of 8, ldb, ldsb of 16.
template <int BM, int BN, int WM, int WN, int STAGES>
constexpr int wq_lds_bytes() {
  return STAGES * (BM * 64 + BN * 16) + 2 * BN * 16;
}

template <int BM, int BN, int WM, int WN, int STAGES, int PANEL>
__global__ __launch_bounds__(64 * WM * WN) void gemm_f16_mxfp4_pp(MxGemmArgs g) {
  constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
  using OpA = PpOperand<BM, 32, 16, true, NW>;
  constexpr int A_BYTES = OpA::BYTES, B_BYTES = BN * 16;
  constexpr int GROUP = 16, SG_BYTES = BN * 16;
  constexpr int BW = BN / 64;  // waves that copy a tile of B (64 rows each), from wave 0 on
  static_assert(NW == 8 && OpA::REM == 0 && BW <= 4 && STAGES <= 4, "copies");

  extern __shared__ __attribute__((aligned(16))) char smem[];
  char* const a_lds = smem;
  char* const b_lds = smem + STAGES * A_BYTES;
  char* const s_lds = b_lds + STAGES * B_BYTES;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int64_t tm, tn;
  tile_of(blockIdx.x, g.tiles_m, g.tiles_n, PANEL, 1, &tm, &tn);
  const int row0 = (int)tm * BM, col0 = (int)tn * BN;
  const int mvalid = min(BM, g.M - row0), nvalid = min(BN, g.N - col0);
  const int nk = g.KB;
  const int kin_last = g.K - (nk - 1) * kMxBlock;

  OpA opa;
  opa.init_copies((const _Float16*)g.A, g.lda, row0, mvalid, kin_last, wave, lane);
  const uint32_t a_lds0 = lds_addr(a_lds) + wave * 1024;
  // Waves 0 .. BW-1 copy 64 rows of B's codes per k-tile, waves 4 .. 4+BW-1 (the other group,
  // which copies less) 64 rows of scales every 16 k-tiles.
  const int part = wave & 3;
  const bool has_b = part < BW;
  const char* const b_base = (const char*)(g.B + (int64_t)(col0 + part * 64) * g.ldb);
  const char* const s_base = (const char*)(g.SB + (int64_t)(col0 + part * 64) * g.ldsb);
  const uint32_t b_off = lane < nvalid - part * 64 ? (uint32_t)(lane * g.ldb) : kOob;
  const uint32_t s_off = lane < nvalid - part * 64 ? (uint32_t)(lane * g.ldsb) : kOob;
  const uint32_t b_dst = lds_addr(b_lds) + part * 1024, s_dst = lds_addr(s_lds) + part * 1024;

  const char* b_next = b_base;  // (a running pointer: 42.9 us against 44.5 for 512 x 4096 x 4096)
  auto copy_tile = [&](int t, auto group) __attribute__((always_inline)) {
    constexpr int G = decltype(group)::value;
    const int slot = t % STAGES;
    const bool last = t == nk - 1;
    const int4v ra = opa.rsrc(t, nk, nk);
    if (G == 1 && t % GROUP == 0 && t < nk && has_b)
      dma_to_lds(make_rsrc(s_base + t, kMaxRange), s_dst + ((t / GROUP) & 1) * SG_BYTES, s_off);
#pragma unroll
    for (int j = 0; j < OpA::LD; ++j)
      dma_to_lds(ra, a_lds0 + slot * A_BYTES + j * NW * 1024, last ? opa.off_last[j] : opa.off[j]);
    if (G == 0 && has_b) dma_to_lds(make_rsrc(b_next, t < nk ? kMaxRange : 0u), b_dst + slot * B_BYTES, b_off);
    b_next += kMxBlockBytes;
  };

  const int wm = wave / WN, wn = wave % WN, lrow = lane & 15, lkg = lane >> 4;
  opa.init_frags(wm * WTM, lane);
  const char* const b_rd = b_lds + (wn * WTN + lrow) * 16 + 4 * lkg;
  const char* const s_rd = s_lds + (wn * WTN + lrow) * 16;

  half8 fa[FM], fb[FN];
  auto read_tile = [&](int t) __attribute__((always_inline)) {
    const char* const As = a_lds + (t % STAGES) * A_BYTES;
    uint32_t w[FN], s[FN];
    const int so = ((t / GROUP) & 1) * SG_BYTES + t % GROUP;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
      w[fn] = *(const TG_LDS uint32_t*)(b_rd + (t % STAGES) * B_BYTES + fn * 256);
      s[fn] = *(const TG_LDS uint8_t*)(s_rd + so + fn * 256);
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) fa[fm] = opa.frag(As, fm, 0);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) fb[fn] = decode8(w[fn], s[fn]);
  };

  float4v acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  auto mma_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
        acc[fm][fn] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[fn], fa[fm], acc[fm][fn], 0, 0, 0);
  };
  // every wave copies at least A's share of a tile (waves 0 .. BW-1 one more)
  constexpr int PT = OpA::LD;
  pingpong_schedule<STAGES, PT, PT, false>(wave / 4, nk, copy_tile, read_tile, mma_tile);

  using ST = StagedTile<WTM, WTN>;
  static_assert(NW * ST::BYTES <= 160 * 1024, "staged tile");
  __syncthreads();
  char* const stage = smem + wave * ST::BYTES;
  if (g.relu != 0)
    ST::template stage<true>(stage, acc, lane);
  else
    ST::template stage<false>(stage, acc, lane);
  ST::wave_fence();
  store_staged<ST, WTM>(stage, lane, g.C + (int64_t)(row0 + wm * WTM) * g.ldc + col0 + wn * WTN, g.ldc,
                        mvalid - wm * WTM, nvalid - wn * WTN, g.vec_c);
}

// ------------------------------------------------------------------------------------
// Few rows (single tokens and small batches): bound by reading the weight once for every 64 rows
// of A, and at these sizes by the latency of a launch and of dependent trips to memory (two up to 16
// rows; four of A's chunks one after another in a run for more than 32 binary16 rows). A
// workgroup owns 16 rows of the weight and up to 64 of A and splits K over its W waves in runs of
// 512 (16 blocks: one 16-byte load of scales per row, four loads of codes), so all of a wave's
// loads of a run are in flight at once; the waves' partial sums are added in wave order. Lane l of
// the weight's fragment holds block l / 16 (of four) of row l % 16, 32 codes.
// 1 x 8192 x 4096: 6.0 us with MXFP4 A, 7.1 with binary16 (a weight of 17.8 MB: 3.0 and 2.5 TB/s,
// launch included); 1 x 8192 x 8192: 10.4 and 13.4, of which 3 are binary16 A's way through LDS and
// the decode; 37 x 3000 x 4096 with binary16 A 9.5, on 188 workgroups.
// Rows of scales that are not padded to 16 bytes cost a little (1 x 8192 x 3000: 3.7 -> 4.6 us, binary16
// 4.7 -> 5.3; 8 x 8192 x 8200: 7.9 -> 10.2, 13.4 -> 16.8; the generic kernel 72 to 273).
// Codes of A come the same way. Binary16 A meets a block's codes in four MFMAs of 8 k per lane,
// step j taking k 32 (l / 16) + 8 j .. + 7 on both sides (any order of k will do that both
// operands share). Loaded straight into that layout, every lane would touch a 64-byte segment
// of its own for 16 bytes of it (13 us for 37 x 3000 x 4096, against 9); so the rows of A are
// loaded 256 contiguous bytes each, four rows per load, and pass through a part of LDS that
// belongs to the wave (no barrier; chunk c of row r at place c ^ r, free of bank conflicts).
// LR: loads that cover the rows of A (4 MT, or one for up to four rows, the others zeros). PADDED: the
// rows of scales lie in whole 16-byte pieces.
template <int MT, int W, int LR, bool F16A, bool PADDED>
__global__ __launch_bounds__(64 * W) void gemm_mxfp4_skinny(MxGemmArgs g) {
  constexpr int A_BYTES = F16A ? MT * 16 * 256 : 0;              // per wave: 16 MT rows of 128 k
  constexpr int P_BYTES = W * MT * 64 * 16;                      // partial sums, in the same place
  extern __shared__ __attribute__((aligned(16))) char smem[];
  static_assert((W * A_BYTES > P_BYTES ? W * A_BYTES : P_BYTES) <= 128 * 1024, "LDS");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lrow = lane & 15, lblk = lane >> 4;
  const int n0 = (int)blockIdx.x * 16, m0 = (int)blockIdx.y * kMxSkinnyTile;
  const int rows = min(g.M - m0, MT * 16);
  const int n = min(n0 + lrow, g.N - 1);  // rows past N read the last one, their sums are dropped
  const uint8_t* const brow = g.B + (int64_t)n * g.ldb + lblk * kMxBlockBytes;
  const uint8_t* const srow = g.SB + (int64_t)n * g.ldsb;
  // The 16 scales of a run, one load; rows that are not padded to 16 bytes have no bytes past KB, so
  // a lane takes its own four of the last run one by one.
  auto run_scales = [&](const uint8_t* row, int kb0) __attribute__((always_inline)) {
    if (PADDED || kb0 + 16 <= g.KB) return load_any<uint4v>(row + kb0);
    uint4v v = {0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (kb0 + 4 * c + lblk < g.KB) v[c] = (uint32_t)row[kb0 + 4 * c + lblk] << (8 * lblk);
    return v;
  };
  const int runs = (g.KB + 15) / 16;
  char* const a_lds = smem + wave * A_BYTES;
  float4v acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};

  if constexpr (F16A) {
    const half8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int i = LR; i < 4 * MT; ++i) *(TG_LDS half8*)(a_lds + i * 1024 + lane * 16) = zero;
  }
  for (int r = wave; r < runs; r += W) {
    const int kb0 = r * 16;
    uint4v w[4];
    const uint4v sv = run_scales(srow, kb0);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      w[c] = (uint4v){0, 0, 0, 0};
      if (kb0 + 4 * c + lblk < g.KB) w[c] = load_any<uint4v>(brow + (int64_t)(kb0 + 4 * c) * kMxBlockBytes);
    }
    // blocks past KB: zero codes, and a finite scale whatever the padding holds
    auto scale_at = [&](const uint4v& s, int c) { return kb0 + 4 * c + lblk < g.KB ? (s[c] >> (8 * lblk)) & 255u : 127u; };
    if constexpr (F16A) {
      // rows 4 i + lane / 16 of A, 16 bytes per lane: AHEAD chunks are loaded before they are used
      // (all four of a run for up to 16 rows)
      constexpr int AHEAD = MT == 1 ? 4 : MT == 2 ? 2 : 1;
      half8 x[AHEAD][LR];
      auto fetch = [&](int c) __attribute__((always_inline)) {
        const int k = (kb0 + 4 * c) * kMxBlock + 8 * lrow;
#pragma unroll
        for (int i = 0; i < LR; ++i) {
          x[c % AHEAD][i] = (half8){0, 0, 0, 0, 0, 0, 0, 0};
          const int m = 4 * i + lblk;
          if (m < rows && k < g.K)  // (any alignment of A, any K)
            x[c % AHEAD][i] = __builtin_bit_cast(half8, load8((const _Float16*)g.A + (int64_t)(m0 + m) * g.lda + k, g.K - k));
        }
      };
#pragma unroll
      for (int c = 0; c < AHEAD; ++c) fetch(c);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int i = 0; i < LR; ++i) {
          const int m = 4 * i + lblk;
          *(TG_LDS half8*)(a_lds + m * 256 + ((lrow ^ (m & 15)) << 4)) = x[c % AHEAD][i];
        }
        StagedTile<16, 64>::wave_fence();
        if (c + AHEAD < 4) fetch(c + AHEAD);
        const uint32_t sb = scale_at(sv, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8 b = decode8(w[c][j], sb);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const half8 a = *(const TG_LDS half8*)(a_lds + (16 * i + lrow) * 256 + (((4 * lblk + j) ^ lrow) << 4));
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a, acc[i], 0, 0, 0);
          }
        }
        StagedTile<16, 64>::wave_fence();
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int m = m0 + min(16 * i + lrow, rows - 1);  // rows past M read the last one
        const uint8_t* const arow = (const uint8_t*)g.A + (int64_t)m * g.lda + (int64_t)(kb0 + lblk) * kMxBlockBytes;
        const uint4v sa = run_scales(g.SA + (int64_t)m * g.ldsa, kb0);
        uint4v a[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          a[c] = (uint4v){0, 0, 0, 0};
          if (kb0 + 4 * c + lblk < g.KB) a[c] = load_any<uint4v>(arow + 4 * c * kMxBlockBytes);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int4v x = __builtin_bit_cast(int4v, a[c]), b = __builtin_bit_cast(int4v, w[c]);
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1), __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1),
              acc[i], 4, 4, 0, (int)scale_at(sv, c), 0, (int)scale_at(sa, c));
        }
      }
    }
  }
  __syncthreads();  // every wave is done with its rows of A
  float4v* const part = (float4v*)smem;
#pragma unroll
  for (int i = 0; i < MT; ++i) *(TG_LDS float4v*)(part + (wave * MT + i) * 64 + lane) = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += W) {
    float4v s = *(const TG_LDS float4v*)(part + i * 64 + lane);
#pragma unroll
    for (int w = 1; w < W; ++w) s += *(const TG_LDS float4v*)(part + (w * MT + i) * 64 + lane);
    const int m = 16 * i + lrow, c = n0 + 4 * lblk;
    if (m >= rows) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < g.N) g.C[(int64_t)(m0 + m) * g.ldc + c + e] = (_Float16)(g.relu ? relu_f(s[e]) : s[e]);
  }
}

// ------------------------------------------------------------------------------------
// Any alignment, stride and K: 128 x 128 tiles, four waves of 64 x 64, one block of 32 k at a
// time through a double-buffered LDS tile filled through registers (unaligned loads). Codes of
// A are decoded without their scale, which multiplies the block's product in float32 together
// with B's (E8M0 scales leave binary16's range); a binary16 A meets the decoded weight. Bound by
// the loads through registers, whose latency one block does not cover: 4096^3 takes 377 us with
// MXFP4 A and 301 with binary16.
template <bool F16A>
__global__ __launch_bounds__(256) void gemm_mxfp4_generic(MxGemmArgs g) {
  constexpr int ROW = 40;  // halves per LDS row: 16-byte aligned, rows spread over the banks
  __shared__ __attribute__((aligned(16))) _Float16 at[2][128 * ROW], bt[2][128 * ROW];
  __shared__ int as[2][128], bs[2][128];  // scale exponents
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row0 = (int)(blockIdx.x / g.tiles_n) * 128, col0 = (int)(blockIdx.x % g.tiles_n) * 128;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64, lrow = lane & 15, lkg = lane >> 4;
  // thread t stages half (t & 1) of row t / 2 of both tiles: 16 values of A, 16 codes of B
  const int sr = tid >> 1, sh = tid & 1;
  const bool a_in = row0 + sr < g.M, b_in = col0 + sr < g.N;
  const int64_t ar = a_in ? row0 + sr : 0, br = b_in ? col0 + sr : 0;
  uint4v av[2];
  uint2v bv;
  uint32_t sav = 127, sbv = 127;
  auto fetch = [&](int kb) {
    if constexpr (F16A) {
      const int k = kb * kMxBlock + 16 * sh;
#pragma unroll
      for (int h = 0; h < 2; ++h) av[h] = load8((const _Float16*)g.A + ar * g.lda + k + 8 * h, a_in ? g.K - k - 8 * h : 0);
    } else {
      const uint2v c = load_any<uint2v>((const uint8_t*)g.A + ar * g.lda + (int64_t)kb * kMxBlockBytes + 8 * sh);
      av[0] = (uint4v){c[0], c[1], 0, 0};
      sav = g.SA[ar * g.ldsa + kb];
    }
    bv = load_any<uint2v>(g.B + br * g.ldb + (int64_t)kb * kMxBlockBytes + 8 * sh);
    sbv = g.SB[br * g.ldsb + kb];
  };
  auto put = [&](int buf) {
    half8 a0, a1;
    if constexpr (F16A) {
      a0 = __builtin_bit_cast(half8, av[0]);
      a1 = __builtin_bit_cast(half8, av[1]);
    } else {
      a0 = decode8(av[0][0], sav == 255 ? 255 : 127);  // a NaN scale makes NaN values
      a1 = decode8(av[0][1], sav == 255 ? 255 : 127);
      if (sh == 0) {
        as[buf][sr] = (int)sav - 127;
        bs[buf][sr] = (int)sbv - 127;
      }
    }
    *(half8*)&at[buf][sr * ROW + 16 * sh] = a0;
    *(half8*)&at[buf][sr * ROW + 16 * sh + 8] = a1;
    *(half8*)&bt[buf][sr * ROW + 16 * sh] = decode8(bv[0], F16A || sbv == 255 ? sbv : 127);
    *(half8*)&bt[buf][sr * ROW + 16 * sh + 8] = decode8(bv[1], F16A || sbv == 255 ? sbv : 127);
  };
  float4v acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = (float4v){0.0f, 0.0f, 0.0f, 0.0f};
  fetch(0);
  put(0);
  __syncthreads();
  for (int kb = 0; kb < g.KB; ++kb) {
    const int buf = kb & 1;
    if (kb + 1 < g.KB) fetch(kb + 1);
    half8 fa[4], fb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa[f] = *(const half8*)&at[buf][(wm + 16 * f + lrow) * ROW + 8 * lkg];
      fb[f] = *(const half8*)&bt[buf][(wn + 16 * f + lrow) * ROW + 8 * lkg];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F16A) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        } else {
          const float4v zero = {0.0f, 0.0f, 0.0f, 0.0f};
          const float4v p = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], zero, 0, 0, 0);
          // the exponents are added first: either scale alone may leave float32's range
          const int sa = as[buf][wm + 16 * i + lrow];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] += __builtin_amdgcn_ldexpf(p[e], sa + bs[buf][wn + 16 * j + 4 * lkg + e]);
        }
      }
    if (kb + 1 < g.KB) put(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = row0 + wm + 16 * i + lrow;
    if (m >= g.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = col0 + wn + 16 * j + 4 * lkg + e;
        if (c < g.N) g.C[(int64_t)m * g.ldc + c] = (_Float16)(g.relu ? relu_f(acc[i][j][e]) : acc[i][j][e]);
      }
  }
}

// Launch of a kernel with more than the default dynamic LDS: the limit is raised once per
// kernel and device.
template <typename K>
hipError_t launch_big(K kern, int lds, std::atomic<uint64_t>& ready, const MxGemmArgs& g, hipStream_t s, int device,
                      dim3 grid, int threads) {
  const uint64_t bit = 1ull << (device & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  hipLaunchKernelGGL(kern, grid, dim3(threads), lds, s, g);
  return hipGetLastError();
}
template <typename K>
hipError_t launch_big(K kern, int lds, std::atomic<uint64_t>& ready, const MxGemmArgs& g, hipStream_t s, int device) {
  return launch_big(kern, lds, ready, g, s, device, dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n)), 512);
}

template <int BM>
hipError_t launch_wq_pp(const MxGemmArgs& g, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  constexpr int ring = wq_lds_bytes<BM, BM, 2, 4, 4>(), st = 8 * StagedTile<BM / 2, BM / 4>::BYTES;
  return launch_big(gemm_f16_mxfp4_pp<BM, BM, 2, 4, 4, 4>, ring > st ? ring : st, ready, g, s, device);
}
template <int BM, int STAGES>
hipError_t launch_mx_small(const MxGemmArgs& g, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  static_assert(kMxSmallLds<BM, STAGES> <= 160 * 1024, "LDS");
  return launch_big(gemm_mxfp4_small<BM, STAGES, 4>, kMxSmallLds<BM, STAGES>, ready, g, s, device);
}
hipError_t launch_mx_256(const MxGemmArgs& g, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  return launch_big(gemm_mxfp4_pp256<4>, kMx256Lds, ready, g, s, device);
}

template <int MT, int W, bool F16A, int LR, bool PADDED>
hipError_t launch_skinny_tile(const MxGemmArgs& g, hipStream_t s, int device) {
  static std::atomic<uint64_t> ready{0};
  constexpr int lds = W * MT * (F16A ? 4096 : 1024);
  const dim3 grid((unsigned)ceil_div(g.N, 16), (unsigned)ceil_div(g.M, kMxSkinnyTile));
  return launch_big(gemm_mxfp4_skinny<MT, W, LR, F16A, PADDED>, lds, ready, g, s, device, grid, 64 * W);
}

// Eight waves, or sixteen for up to 16 rows where K has more than eight runs of 512 (every run
// of a wave after its first waits for memory again; more rows need the registers, and so do 5 to 16
// binary16 rows beside scales taken one by one).
template <bool F16A, bool PADDED>
hipError_t launch_skinny(const MxGemmArgs& g, hipStream_t s, int device) {
  const bool deep = g.KB > 8 * 16;
  switch (g.M >= kMxSkinnyTile ? 4 : (g.M + 15) / 16) {
    case 1:
      if (F16A && g.M <= 4)
        return deep ? launch_skinny_tile<1, 16, F16A, 1, PADDED>(g, s, device) : launch_skinny_tile<1, 8, F16A, 1, PADDED>(g, s, device);
      return deep ? launch_skinny_tile<1, F16A && !PADDED ? 8 : 16, F16A, 4, PADDED>(g, s, device)
                  : launch_skinny_tile<1, 8, F16A, 4, PADDED>(g, s, device);
    case 2: return launch_skinny_tile<2, 8, F16A, 8, PADDED>(g, s, device);
    case 3: return launch_skinny_tile<3, 8, F16A, 12, PADDED>(g, s, device);
    default: return launch_skinny_tile<4, 8, F16A, 16, PADDED>(g, s, device);
  }
}
template <bool F16A>
hipError_t launch_skinny(const MxGemmArgs& g, hipStream_t s, int device) {
  auto padded = [](const uint8_t* S, int64_t lds) { return ((reinterpret_cast<uintptr_t>(S) | (uintptr_t)lds) & 15) == 0; };
  return padded(g.SB, g.ldsb) && (F16A || padded(g.SA, g.ldsa)) ? launch_skinny<F16A, true>(g, s, device)
                                                              : launch_skinny<F16A, false>(g, s, device);
}

}  // namespace

hipError_t launch_mxfp4(int cfg, bool f16_a, const MxGemmArgs& args, hipStream_t s, int device) {
  MxGemmArgs g = args;
  g.tiles_m = (int)ceil_div(g.M, mx_tile_m(cfg));
  g.tiles_n = (int)ceil_div(g.N, mx_tile_n(cfg));
  switch (cfg) {
    case kMxSkinny: return f16_a ? launch_skinny<true>(g, s, device) : launch_skinny<false>(g, s, device);
    case kMx128: return f16_a ? launch_wq_pp<128>(g, s, device) : launch_mx_small<128, 4>(g, s, device);
    case kMx64: return f16_a ? hipErrorNotSupported : launch_mx_small<64, 6>(g, s, device);
    case kMx256: return f16_a ? launch_wq_pp<256>(g, s, device) : launch_mx_256(g, s, device);
    default: break;
  }
  const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n));
  if (f16_a)
    hipLaunchKernelGGL(gemm_mxfp4_generic<true>, grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL(gemm_mxfp4_generic<false>, grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_quant_mxfp4(const MxQuantArgs& q, hipStream_t s) {
  if (q.QT != nullptr) {
    const int64_t tiles = ceil_div(q.R, 256) * ceil_div(q.K, 128);
    if (q.Q != nullptr)
      hipLaunchKernelGGL(quant_mxfp4_cols<true>, dim3((unsigned)tiles), dim3(256), 0, s, q);
    else
      hipLaunchKernelGGL(quant_mxfp4_cols<false>, dim3((unsigned)tiles), dim3(256), 0, s, q);
  } else {
    const int64_t blocks = (int64_t)q.R * ceil_div(q.K, kMxBlock);
    hipLaunchKernelGGL(quant_mxfp4_rows<2>, dim3((unsigned)ceil_div(blocks, 128)), dim3(256), 0, s, q);
  }
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const MxDequantArgs& q, hipStream_t s) {
  const int64_t blocks = (int64_t)q.R * ceil_div(q.K, kMxBlock);
  hipLaunchKernelGGL(dequant_mxfp4_rows<2>, dim3((unsigned)ceil_div(blocks, 128)), dim3(256), 0, s, q);
  return hipGetLastError();
}

}  // namespace tgemm
