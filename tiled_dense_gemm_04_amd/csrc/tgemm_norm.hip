// tgemm_norm.hip -- gfx950 kernels of the root-mean-square norm with the residual's addition, its
// output in binary16 or in E4M3 codes with a scale per 1 x 128 block, and its gradient.
//
//   h = round(x + r) to the residual's type (h = x without one), rstd = 1 / sqrt(mean h^2 + eps),
//   y = h rstd w;  codes of a block: s = max |y| / 448, q = E4M3(y / s).
//   Backward, xhat = h rstd:  dx = rstd (w dy - xhat mean(w dy xhat)) + dh,  dw = sum_rows dy xhat.
// h is the value that is stored, so that the backward pass, which reads it, is the gradient of what
// was computed; y stays in float32 until its one rounding (the codes are not made from a rounded
// binary16 y). Every sum is float32. Both passes are bound by memory: a row is read once, held in
// the registers of 16 to 1024 threads, eight consecutive values a chunk, and written once.
#include "tgemm_device.h"
#include "tgemm_norm.h"
#include "tgemm_rows.h"

namespace tgemm {
namespace {

// N sums over the TPR threads of a row (up to 64: lanes of one wave; else the workgroup, every thread
// adding the waves' sums in wave order). `lds` holds a float per wave and sum; a slow wave may still read
// it when the call returns, so calls that follow each other alternate between two arrays.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[N]) {
#pragma unroll
  for (int o = 1; o < (TPR < 64 ? TPR : 64); o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o, 64);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) lds[threadIdx.x >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll 8
    for (int w = 0; w < TPR / 64; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += lds[w][i];
  }
}

// Two floats to two E4M3 codes in the low or high half of a word (round to nearest even).
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b, uint32_t old) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
}

// Codes and scale of a lane's eight values of a 1 x 128 block (16 neighbouring lanes). Magnitudes
// order like their bit patterns, infinities and NaN at the top: such a block gets a NaN scale and
// zero codes, so that the products it goes to are NaN. A block below 2^-100 counts as zeros (its
// scale's reciprocal would leave float32).
__device__ __forceinline__ float block_codes(const float (&y)[8], uint2v& codes) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(y[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 16));
  codes = (uint2v){0u, 0u};
  if (m >= 0x7F800000u) return __builtin_nanf("");
  if (m < 0x0D800000u) return 1.0f;  // 2^-100
  const float s = __uint_as_float(m) / 448.0f, r = 1.0f / s;
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // y / s: the product with the reciprocal, corrected once by its exact residual
    const float q0 = y[e] * r;
    q[e] = __builtin_fmaf(__builtin_fmaf(-q0, s, y[e]), r, q0);
  }
  codes[0] = e4m3_pair<true>(q[2], q[3], e4m3_pair<false>(q[0], q[1], 0u));
  codes[1] = e4m3_pair<true>(q[6], q[7], e4m3_pair<false>(q[4], q[5], 0u));
  return s;
}

// ------------------------------------------------------------------------------------
// Forward. TPR threads a row, CH chunks of eight values a thread: thread t holds chunks t + i TPR,
// so a 1 x 128 block is 16 neighbouring lanes. The residual, x and the weight of a row are all in
// flight before the one reduction. 16384 x 4096 with a binary16 residual: 99 us (5.4 TB/s) to binary16, 87
// to codes (5.4), where a copy of 1 GiB reaches 5.2; 4095 x 3000 with a float32 one 29 (5.1); one row of
// 4096 3.5 and 4.1 with its launch.
template <int TPR, int CH, int RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_rows(NormArgs g) {
  __shared__ float lds[TPR > 64 ? TPR / 64 : 1][1];
  constexpr int RPG = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPG + threadIdx.x / TPR;
  const bool live = row < g.R;
  const int64_t r = live ? row : g.R - 1;
  float h[CH][8], w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k = 8 * (t + i * TPR), n = g.K - k;
    half8 x = load_half8(g.X + r * g.ldx + k, k, n);
    if constexpr (RES == kResF32) load_float8((const float*)g.Rin + r * g.ldr + k, k, n, h[i]);
    if constexpr (RES == kResF16) {
      const half8 a = load_half8((const _Float16*)g.Rin + r * g.ldr + k, k, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = (float)a[e];
    }
    if (g.w_f32) {
      load_float8((const float*)g.W + k, k, n, w[i]);
    } else {
      const half8 a = load_half8((const _Float16*)g.W + k, k, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = (float)a[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = RES == kResNone ? (float)x[e] : h[i][e] + (float)x[e];
  }
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k = 8 * (t + i * TPR), n = g.K - k;
    if constexpr (RES == kResF16) {
      half8 a;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = (_Float16)h[i][e];
        h[i][e] = (float)a[e];
      }
      if (live && g.Rout != nullptr) store_half8((_Float16*)g.Rout + r * g.ldro + k, a, n);
    }
    if constexpr (RES == kResF32) {
      if (live && g.Rout != nullptr) store_float8((float*)g.Rout + r * g.ldro + k, h[i], n);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[0] = __builtin_fmaf(h[i][e], h[i][e], ss[0]);
  }
  row_sums<TPR>(ss, lds);
  const float rstd = 1.0f / sqrtf(ss[0] / (float)g.K + g.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k = 8 * (t + i * TPR), n = g.K - k;
    float y[8];
    half8 a;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = h[i][e] * rstd * w[i][e];
      a[e] = (_Float16)y[e];
    }
    if (live && g.Y != nullptr) store_half8(g.Y + r * g.ldy + k, a, n);
    if (g.Q != nullptr) {
      uint2v codes;
      const float s = block_codes(y, codes);  // (zeros past K)
      if (live) store_bytes8(g.Q + r * g.ldq + k, codes, n);
      if (live && n > 0 && t % 16 == 0) g.S[r * g.KB + k / kFp8Block] = s;
    }
  }
}

// ------------------------------------------------------------------------------------
// Backward; a row's rstd is computed again beside the other sum it needs, from the row that is there
// anyway. A workgroup takes rows blockIdx.x, + gridDim.x, ... (times its rows at once); a thread
// keeps its columns' weights and its sums of dw in registers over all of them, and the sums leave
// as one row of partial sums per workgroup, added in a fixed order by norm_weight_grad. With that kernel
// 8192 x 8192 takes 104 us in a loop (5.2 TB/s) and 116 after other work; in a loop 16384 x 4096 110,
// 16384 x 2048 52, 131072 x 128 18.5.
template <int TPR, int CH, bool H32>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_grad_rows(NormGradArgs g) {
  __shared__ float lds[2][TPR > 64 ? TPR / 64 : 1][2];
  constexpr int RPG = TPR < 256 ? 256 / TPR : 1;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int k = 8 * (t + i * TPR), n = g.K - k;
    if (g.w_f32) {
      load_float8((const float*)g.W + k, k, n, w[i]);
    } else {
      const half8 a = load_half8((const _Float16*)g.W + k, k, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = (float)a[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  const float inv_k = 1.0f / (float)g.K;
  int parity = 0;
  for (int64_t first = (int64_t)blockIdx.x * RPG; first < g.R; first += (int64_t)gridDim.x * RPG, parity ^= 1) {
    const bool live = first + sub < g.R;
    const int64_t r = live ? first + sub : g.R - 1;
    // (a column of the row's own: what follows from it, conditions above all, would spill if kept over the loop)
    int column = t;
    asm volatile("" : "+v"(column));
    half8 dy[CH];
    float h[CH][8];
    float sum[2] = {0.0f, 0.0f};  // of h^2 and of w dy h
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int k = 8 * (column + i * TPR), n = g.K - k;
      dy[i] = load_half8(g.dY + r * g.lddy + k, k, n);
      if constexpr (H32) {
        load_float8((const float*)g.H + r * g.ldh + k, k, n, h[i]);
      } else {
        const half8 a = load_half8((const _Float16*)g.H + r * g.ldh + k, k, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = (float)a[e];
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] = __builtin_fmaf(h[i][e], h[i][e], sum[0]);
        sum[1] = __builtin_fmaf((float)dy[i][e] * w[i][e], h[i][e], sum[1]);
      }
    row_sums<TPR>(sum, lds[parity]);
    const float rstd = 1.0f / sqrtf(sum[0] * inv_k + g.eps), c = sum[1] * inv_k * rstd;
    if (live) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int k = 8 * (column + i * TPR), n = g.K - k;
        float dx[8], dh[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[e] = 0.0f;
        if (g.dH != nullptr) {
          if constexpr (H32) {
            load_float8((const float*)g.dH + r * g.lddh + k, k, n, dh);
          } else {
            const half8 a = load_half8((const _Float16*)g.dH + r * g.lddh + k, k, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) dh[e] = (float)a[e];
          }
        }
        half8 a;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xhat = h[i][e] * rstd;
          dw[i][e] = __builtin_fmaf((float)dy[i][e], xhat, dw[i][e]);
          dx[e] = __builtin_fmaf(rstd, __builtin_fmaf(-xhat, c, (float)dy[i][e] * w[i][e]), dh[e]);
          a[e] = (_Float16)dx[e];
        }
        store_half8(g.dX + r * g.lddx + k, a, n);
        if (g.dR != nullptr) {
          if constexpr (H32)
            store_float8((float*)g.dR + r * g.lddr + k, dx, n);
          else
            store_half8((_Float16*)g.dR + r * g.lddr + k, a, n);
        }
      }
    }
  }
  if (g.dW == nullptr) return;
  float* const out = g.parts + (int64_t)blockIdx.x * g.K;
  if constexpr (RPG > 1) {  // the waves' rows are joined, in wave order
    __shared__ float join[RPG][CH * 8 * TPR];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) join[sub][8 * (t + i * TPR) + e] = dw[i][e];
    __syncthreads();
    for (int k = threadIdx.x; k < g.K; k += 256) {
      float v = join[0][k];
#pragma unroll
      for (int w = 1; w < RPG; ++w) v += join[w][k];
      out[k] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) store_float8(out + 8 * (t + i * TPR), dw[i], g.K - 8 * (t + i * TPR));
  }
}

// dw from the partial sums: 64 columns per workgroup, wave w adds rows w, w + 16, ...; the waves'
// sums are added in wave order.
__global__ __launch_bounds__(1024) void norm_weight_grad(NormGradArgs g) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = (int)blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (k < g.K) {
#pragma unroll 16
    for (int p = wave; p < g.groups; p += 16) v += g.parts[(int64_t)p * g.K + k];
  }
  lds[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || k >= g.K) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) v += lds[w][lane];
  if (g.w_f32)
    ((float*)g.dW)[k] = v;
  else
    ((_Float16*)g.dW)[k] = (_Float16)v;
}

// Threads per row and chunks per thread for rows of K values: NORM_SHAPE(TPR, CH).
#define TGEMM_NORM_SHAPES(NORM_SHAPE, K)       \
  if (K <= 128) return NORM_SHAPE(16, 1);      \
  if (K <= 256) return NORM_SHAPE(32, 1);      \
  if (K <= 512) return NORM_SHAPE(64, 1);      \
  if (K <= 1024) return NORM_SHAPE(64, 2);     \
  if (K <= 2048) return NORM_SHAPE(256, 1);    \
  if (K <= 4096) return NORM_SHAPE(256, 2);    \
  if (K <= 8192) return NORM_SHAPE(512, 2);    \
  return NORM_SHAPE(1024, 2);

template <int TPR, int CH, int RES>
hipError_t launch_rows(const NormArgs& g, hipStream_t s) {
  constexpr int threads = TPR < 256 ? 256 : TPR, rpg = threads / TPR;
  hipLaunchKernelGGL((rmsnorm_rows<TPR, CH, RES>), dim3((unsigned)ceil_div(g.R, rpg)), dim3(threads), 0, s, g);
  return hipGetLastError();
}
template <int RES>
hipError_t launch_forward(const NormArgs& g, hipStream_t s) {
#define TGEMM_NORM_LAUNCH(TPR, CH) (launch_rows<TPR, CH, RES>(g, s))
  // Six waves of one chunk (a row's threads all busy, but a third fewer rows in flight) instead of four waves of two,
  // where a residual is written beside y. Rows of 2560, 2816 and 3064 values, four and six waves, us:
  //   float32 residual      4095 rows 28.4 27.5, 31.1 29.5, 34.8 32.5;  16384 92.9 90.2, 103.5 99.4, 117.4 110.7
  //   and codes             4095      26.9 26.6, 29.8 28.5, 32.5 31.2;  16384 86.7 85.3, 95.9 93.6, 109.4 105.0
  //   binary16 residual     4095      15.9 15.0, 18.3 18.1, 21.1 21.0;  16384 62.7 60.5, 69.3 66.5, 77.1 73.1
  //   and codes (not taken) 4095      16.8 16.2, 18.3 17.6, 19.8 19.9;  16384 59.0 64.0, 63.2 67.6, 70.2 70.8
  //   none (not taken)      4095      10.3 11.0, 10.9 11.5, 11.4 11.9;  16384 36.0 42.9, 38.4 45.8, 42.3 47.2
  // 2100 rows with a float32 residual 17.7 17.4, 19.0 18.5, 21.2 20.2, but 1800 15.0 15.4, 16.0 16.3, 17.9 18.0, and
  // 16384 x 2304 with a binary16 one 57.8 57.8. (The runtime takes fewer than 2^32 threads.)
  if constexpr (RES != kResNone) {
    if ((RES == kResF32 || g.Q == nullptr) && g.K >= 2560 && g.K <= 384 * 8 && g.R >= 2048 && g.R <= (1 << 23))
      return launch_rows<384, 1, RES>(g, s);
  }
  TGEMM_NORM_SHAPES(TGEMM_NORM_LAUNCH, g.K)
#undef TGEMM_NORM_LAUNCH
}

template <int TPR, int CH, bool H32>
hipError_t launch_grad_rows(const NormGradArgs& g, hipStream_t s) {
  constexpr int threads = TPR < 256 ? 256 : TPR;
  hipLaunchKernelGGL((rmsnorm_grad_rows<TPR, CH, H32>), dim3((unsigned)g.groups), dim3(threads), 0, s, g);
  return hipGetLastError();
}
template <bool H32>
hipError_t launch_grad(const NormGradArgs& g, hipStream_t s) {
#define TGEMM_NORM_LAUNCH(TPR, CH) (launch_grad_rows<TPR, CH, H32>(g, s))
  TGEMM_NORM_SHAPES(TGEMM_NORM_LAUNCH, g.K)
#undef TGEMM_NORM_LAUNCH
}

}  // namespace

// Sixteen waves a compute unit (half of them: 16384 x 2048 68 us instead of 52, 16384 x 4096 117 instead
// of 110), each group at least twice the rows it holds at once (512 x 4096: 14.4 us with one row a group,
// 11.8 with two, 14.3 with four).
int norm_grad_groups(int64_t R, int64_t K) {
  const int64_t threads = norm_row_threads(K), group = threads < 256 ? 256 : threads;
  const int64_t want = ceil_div(R, 2 * (group / threads)), most = 256 * 1024 / group;
  return (int)(want < most ? want : most);
}

hipError_t launch_rmsnorm(const NormArgs& g, int residual, hipStream_t s) {
  switch (residual) {
    case kResF16: return launch_forward<kResF16>(g, s);
    case kResF32: return launch_forward<kResF32>(g, s);
    default: return launch_forward<kResNone>(g, s);
  }
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& g, bool h_f32, hipStream_t s) {
  const hipError_t e = g.groups == 0 ? hipSuccess : h_f32 ? launch_grad<true>(g, s) : launch_grad<false>(g, s);
  if (e != hipSuccess || g.dW == nullptr) return e;
  hipLaunchKernelGGL(norm_weight_grad, dim3((unsigned)ceil_div(g.K, 64)), dim3(1024), 0, s, g);
  return hipGetLastError();
}

}  // namespace tgemm
