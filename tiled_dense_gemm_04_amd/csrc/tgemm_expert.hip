// tgemm_expert.hip -- gfx950 kernels that bring tokens to their experts and back: a stable counting
// sort of the slots by expert, rows gathered into sorted order, and the weighted sum of a token's
// rows, with its gradient.
//
//   slot s = t k + j, id[s] in [0, E) or anything else for no expert;
//   offsets[e] = slots with an id below e;  place[s] = offsets[id[s]] + earlier slots of that id;
//   gather:  dst[place[s]] = src[t];   combine:  dst[t] = sum_j w[s] src[place[s]];
//   combine's gradient:  dY[place[s]] = w[s] dout[t],  dw[s] = <dout[t], Y[place[s]]>.
// The gradient of gather is combine without weights. No atomics: every result is the same in every
// run. An index outside its range counts as no row, whatever wrote it.
#include "tgemm_expert.h"
#include "tgemm_rows.h"

namespace tgemm {
namespace {

// The class of slot s: its expert, or E where it has none.
template <bool I64>
__device__ __forceinline__ int slot_class(const ExpertSortArgs& g, int s) {
  int64_t at = s;
  if (g.ldi != g.k) {
    const int t = s / g.k;
    at = (int64_t)t * g.ldi + (s - t * g.k);
  }
  if constexpr (I64) {
    const uint64_t v = ((const uint64_t*)g.ids)[at];
    return v < (uint64_t)g.experts ? (int)v : g.experts;
  } else {
    const uint32_t v = ((const uint32_t*)g.ids)[at];
    return v < (uint32_t)g.experts ? (int)v : g.experts;
  }
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// ------------------------------------------------------------------------------------
// Up to kSortOneLaunch slots: workgroup c owns class c (c = E: the slots of no expert, which go last
// with order and place -1). A wave looks through a contiguous part of the slots, 64 at a time, and
// keeps the ballots of its class in its lanes (lane i that of step i), so the ids are read once and
// each lane then places the few slots of its ballot; the waves' counts meet in LDS. The ids come from L2 E + 1 times over, which for these sizes costs
// less than a second launch.
constexpr int kSortAhead = 16;  // loads in flight
template <bool I64>
__global__ __launch_bounds__(1024) void expert_sort_small(ExpertSortArgs g) {
  __shared__ int wave_eq[16], wave_lt[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int c = blockIdx.x;
  const int steps = (g.n + 64 * waves - 1) / (64 * waves);  // at most 64
  const int s0 = wave * steps * 64;
  uint64_t mine = 0;
  int eq = 0, lt = 0;
  for (int i = 0; i < steps; i += kSortAhead) {
    int v[kSortAhead];
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      const int s = s0 + 64 * (i + q) + lane;
      v[q] = kMaxExperts + 1;
      if (i + q < steps && s < g.n) v[q] = slot_class<I64>(g, s);
    }
#pragma unroll
    for (int q = 0; q < kSortAhead; ++q) {
      const uint64_t hit = __builtin_amdgcn_ballot_w64(v[q] == c);
      lt += __builtin_popcountll(__builtin_amdgcn_ballot_w64(v[q] < c));
      eq += __builtin_popcountll(hit);
      if (lane == i + q) mine = hit;
    }
  }
  if (lane == 0) {
    wave_eq[wave] = eq;
    wave_lt[wave] = lt;
  }
  __syncthreads();
  int first = 0, row = 0;
  for (int w = 0; w < waves; ++w) {
    first += wave_lt[w];
    if (w < wave) row += wave_eq[w];
  }
  if (threadIdx.x == 0) g.offsets[c] = first;
  // lane i places the slots of step i: those of the steps before come first
  int incl = __builtin_popcountll(mine);
  const int own = incl;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  int p = first + row + incl - own;
  for (; mine != 0; mine &= mine - 1, ++p) {
    const int s = s0 + 64 * lane + __builtin_ctzll(mine);
    g.place[s] = c < g.experts ? p : -1;
    g.order[p] = c < g.experts ? s : -1;
  }
}

// ------------------------------------------------------------------------------------
// More slots: each of kSortSegments waves counts a contiguous segment by class (a counter per class
// in LDS) and leaves every slot's rank in its segment in place[]; then each wave finds where its
// segment's classes start from all segments' counts and writes the places.
constexpr int kSortWaves = 4;

template <bool I64>
__global__ __launch_bounds__(64 * kSortWaves) void expert_sort_count(ExpertSortArgs g, int steps, int bits) {
  __shared__ int count[kSortWaves][kMaxExperts + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg = (int)blockIdx.x * kSortWaves + wave;
  for (int e = lane; e <= g.experts; e += 64) count[wave][e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)seg * steps * 64;
  for (int i0 = 0; i0 < steps; i0 += 8) {  // eight loads in flight
    int v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t s = s0 + 64 * (i0 + q) + lane;
      v[q] = -1;
      if (i0 + q < steps && s < g.n) v[q] = slot_class<I64>(g, (int)s);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // lanes of the same class, bit by bit
      uint64_t same = __builtin_amdgcn_ballot_w64(v[q] >= 0);
      if (same == 0) break;
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __builtin_amdgcn_ballot_w64((v[q] >> b) & 1);
        same &= (v[q] >> b) & 1 ? set : ~set;
      }
      if (v[q] >= 0) {
        const int below = lanes_below(same), base = count[wave][v[q]];
        g.place[s0 + 64 * (i0 + q) + lane] = base + below;
        // (the wave's reads above come before this write: LDS runs a wave's accesses in order)
        if (below == 0) count[wave][v[q]] = base + __builtin_popcountll(same);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    }
  }
  for (int e = lane; e <= g.experts; e += 64) g.counts[(int64_t)seg * (g.experts + 1) + e] = count[wave][e];
}

template <bool I64>
__global__ __launch_bounds__(64 * kSortWaves) void expert_sort_place(ExpertSortArgs g, int segments, int steps) {
  __shared__ int start[kSortWaves][kMaxExperts + 1];
  __shared__ int total[kMaxExperts + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg0 = (int)blockIdx.x * kSortWaves, classes = g.experts + 1;
  // column sums: of all segments, and of those before each of this workgroup's
  for (int e = threadIdx.x; e < classes; e += 64 * kSortWaves) {
    int before = 0, all = 0;
    for (int q0 = 0; q0 < segments; q0 += 16) {  // (a multiple of 16)
      int c[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) c[q] = g.counts[(int64_t)(q0 + q) * classes + e];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        if (q0 + q < seg0) before += c[q];
        all += c[q];
      }
    }
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      start[w][e] = before;
      before += g.counts[(int64_t)(seg0 + w) * classes + e];
    }
    total[e] = all;
  }
  __syncthreads();
  // exclusive sums of the classes' totals, by the first wave: lane l over classes l * c .. + c
  if (wave == 0) {
    const int per = (classes + 63) / 64, e0 = lane * per, e1 = min(e0 + per, classes);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += total[e];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    int at = incl - sum;
    for (int e = e0; e < e1; ++e) {
      const int n = total[e];
      total[e] = at;
      if (blockIdx.x == 0) g.offsets[e] = at;
      at += n;
    }
  }
  __syncthreads();
  const int64_t s0 = (int64_t)(seg0 + wave) * steps * 64;
  for (int i = 0; i < steps; i += 4) {  // four slots in flight
    int v[4], rank[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t s = s0 + 64 * (i + q) + lane;
      v[q] = -1;
      if (i + q < steps && s < g.n) {
        v[q] = slot_class<I64>(g, (int)s);
        rank[q] = g.place[s];
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int s = (int)(s0 + 64 * (i + q) + lane);
      if (v[q] < 0) continue;
      const int p = total[v[q]] + start[wave][v[q]] + rank[q];
      g.place[s] = v[q] < g.experts ? p : -1;
      g.order[p] = v[q] < g.experts ? s : -1;
    }
  }
}

// ------------------------------------------------------------------------------------
// Rows. A thread holds eight columns of a token: reads them once and writes them to every place of
// the token (gather), or sums the token's rows there in float32, choice by choice (combine). Bound
// by memory. The workgroups past `main` zero the rows behind the last one in use.
__device__ __forceinline__ int rows_in_use(const ExpertRowsArgs& g) {
  const int n = g.offsets[g.experts];
  return n < 0 ? 0 : n < g.rows ? n : g.rows;
}
constexpr int kRestGroups = 64;
__device__ __forceinline__ void zero_rest_rows(const ExpertRowsArgs& g, int part, uint32_t cpr) {
  const half8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int r = rows_in_use(g) + part; r < g.rows; r += kRestGroups)
    for (uint32_t c = threadIdx.x; c < cpr; c += 256)
      store_half8(g.dst + (int64_t)r * g.ldd + 8 * c, zero, g.H - 8 * (int)c);
}

__global__ __launch_bounds__(256) void expert_gather(ExpertRowsArgs g, uint32_t main) {
  const uint32_t cpr = ((uint32_t)g.H + 7) / 8;
  if (blockIdx.x >= main) return zero_rest_rows(g, (int)(blockIdx.x - main), cpr);
  const uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= (uint64_t)g.tokens * cpr) return;
  const uint32_t t = (uint32_t)u / cpr, c = (uint32_t)u - t * cpr;  // the host keeps the chunks below 2^32
  const int n = g.H - 8 * (int)c;
  const half8 x = load_half8(g.src + (int64_t)t * g.lds_ + 8 * c, n);
  const int* const place = g.place + (int64_t)t * g.k;
  for (int j0 = 0; j0 < g.k; j0 += 4) {  // four places before the first store
    int p[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] = j0 + q < g.k ? place[j0 + q] : -1;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if ((unsigned)p[q] < (unsigned)g.rows) store_half8(g.dst + (int64_t)p[q] * g.ldd + 8 * c, x, n);
  }
}

__device__ __forceinline__ float slot_weight(const ExpertRowsArgs& g, int64_t s) {
  return g.weights == nullptr ? 1.0f : g.w_f32 ? ((const float*)g.weights)[s] : (float)((const _Float16*)g.weights)[s];
}

__global__ __launch_bounds__(256) void expert_combine(ExpertRowsArgs g) {
  const uint32_t cpr = ((uint32_t)g.H + 7) / 8;
  const uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= (uint64_t)g.tokens * cpr) return;
  const uint32_t t = (uint32_t)u / cpr, c = (uint32_t)u - t * cpr;
  const int n = g.H - 8 * (int)c;
  const int64_t s0 = (int64_t)t * g.k;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
  for (int j0 = 0; j0 < g.k; j0 += 4) {  // four rows in flight
    half8 y[4];
    float w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int p = j0 + q < g.k ? g.place[s0 + j0 + q] : -1;
      const bool live = (unsigned)p < (unsigned)g.rows;
      y[q] = (half8){0, 0, 0, 0, 0, 0, 0, 0};
      w[q] = 0.0f;
      if (live) {
        y[q] = load_half8(g.src + (int64_t)p * g.lds_ + 8 * c, n);
        w[q] = slot_weight(g, s0 + j0 + q);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(w[q], (float)y[q][e], sum[e]);
  }
  half8 o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = (_Float16)sum[e];
  store_half8(g.dst + (int64_t)t * g.ldd + 8 * c, o, n);
}

// A wave per slot: its row of dY is written and its product with Y's summed in one pass (a token's
// slots are neighbouring waves, which share dout's row in the caches).
__global__ __launch_bounds__(256) void expert_combine_grad(ExpertRowsArgs g, uint32_t main) {
  const uint32_t cpr = ((uint32_t)g.H + 7) / 8;
  if (blockIdx.x >= main) return zero_rest_rows(g, (int)(blockIdx.x - main), cpr);
  const int lane = threadIdx.x & 63;
  const int64_t s = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (s >= (int64_t)g.tokens * g.k) return;
  const int64_t t = s / g.k;
  const int p = g.place[s];
  float dot = 0.0f;
  if ((unsigned)p < (unsigned)g.rows) {
    const float w = slot_weight(g, s);
    const _Float16* const d = g.src + t * g.lds_;
    const _Float16* const y = g.aux + (int64_t)p * g.lda;
    _Float16* const o = g.dst + (int64_t)p * g.ldd;
#pragma unroll 4
    for (uint32_t c = lane; c < cpr; c += 64) {
      const int n = g.H - 8 * (int)c;
      const half8 a = load_half8(d + 8 * c, n), b = g.dweights != nullptr ? load_half8(y + 8 * c, n) : a;
      half8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (_Float16)(w * (float)a[e]);
        dot = __builtin_fmaf((float)a[e], (float)b[e], dot);
      }
      if (g.dst != nullptr) store_half8(o + 8 * c, v, n);
    }
  }
  if (g.dweights == nullptr) return;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o, 64);
  if (lane != 0) return;
  if (g.w_f32)
    ((float*)g.dweights)[s] = dot;
  else
    ((_Float16*)g.dweights)[s] = (_Float16)dot;
}

template <bool I64>
hipError_t launch_sort(const ExpertSortArgs& g, hipStream_t s) {
  if (g.n <= kSortOneLaunch) {
    // about four steps of 64 slots per wave, up to 16 waves
    const int want = (g.n + 255) / 256, waves = want < 1 ? 1 : want > 16 ? 16 : want;
    hipLaunchKernelGGL(expert_sort_small<I64>, dim3((unsigned)g.experts + 1), dim3(64 * waves), 0, s, g);
    return hipGetLastError();
  }
  // about 1024 slots a segment
  const int64_t want = ceil_div(g.n, 1024 * 16) * 16;
  const int segments = (int)(want < kSortSegments ? want : kSortSegments);
  const int steps = (int)ceil_div(g.n, (int64_t)segments * 64);
  int bits = 1;
  while ((g.experts >> bits) != 0) ++bits;
  const dim3 grid(segments / kSortWaves);
  hipLaunchKernelGGL(expert_sort_count<I64>, grid, dim3(64 * kSortWaves), 0, s, g, steps, bits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(expert_sort_place<I64>, grid, dim3(64 * kSortWaves), 0, s, g, segments, steps);
  return hipGetLastError();
}

uint32_t chunk_groups(const ExpertRowsArgs& g) { return (uint32_t)ceil_div((int64_t)g.tokens * ceil_div(g.H, 8), 256); }

}  // namespace

hipError_t launch_expert_sort(const ExpertSortArgs& g, hipStream_t s) {
  return g.ids_i64 ? launch_sort<true>(g, s) : launch_sort<false>(g, s);
}

hipError_t launch_expert_gather(const ExpertRowsArgs& g, hipStream_t s) {
  const uint32_t main = chunk_groups(g), all = main + (g.offsets != nullptr ? kRestGroups : 0);
  if (all == 0) return hipSuccess;
  hipLaunchKernelGGL(expert_gather, dim3(all), dim3(256), 0, s, g, main);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const ExpertRowsArgs& g, hipStream_t s) {
  hipLaunchKernelGGL(expert_combine, dim3(chunk_groups(g)), dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_expert_combine_grad(const ExpertRowsArgs& g, hipStream_t s) {
  const uint32_t main = (uint32_t)ceil_div((int64_t)g.tokens * g.k, 4);
  const uint32_t all = main + (g.offsets != nullptr && g.dst != nullptr ? kRestGroups : 0);
  if (all == 0) return hipSuccess;
  hipLaunchKernelGGL(expert_combine_grad, dim3(all), dim3(256), 0, s, g, main);
  return hipGetLastError();
}

}  // namespace tgemm
