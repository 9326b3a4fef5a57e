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
// Sorting. A workgroup owns a chunk of consecutive slots, each of its waves a contiguous segment of it
// in steps of 64. The waves count their classes in LDS (integer atomics: the same counts in any order);
// from the slots of each class in the chunks before and of the classes before follows where each
// wave's first slot of a class goes, and a second pass over the segment hands out the places: lanes of
// one class are found bit by bit with ballots. place is written in whole lines, by the slots' own
// workgroup (written by classes, in pieces of a line from every XCD, it took 21 us for 4095 x 8 slots
// of 64 experts after other work, 10 in a loop).
//   One launch, up to kSortOneLaunch slots: every workgroup counts the other chunks' slots for itself.
//   Two, for more: the chunks' counts go through the workspace.
// Bound by the latency of dependent steps. After other work (ids and results out of the caches): 32 slots
// 5.0 us, 4096 7.9, 8192 9.2 in one launch, 9.6, 12.7 and 13.0 in two; 16384 14.0 and 13.1, 32760 23.7 and
// 13.3; 65536 12 to 17 (8 to 256 experts), 2^20 33.
constexpr int kSortWaves = 8, kSortThreads = 64 * kSortWaves;
struct SortCounts {
  int wave[kSortWaves][kMaxExperts + 1];
  int before[kMaxExperts + 1], all[kMaxExperts + 1];  // slots of a class in the chunks before, and in all
};

__device__ __forceinline__ void count_slot(int* p) { __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP); }

// Counts slots [s0, s1), one in `stride` from s0 on, by class; eight loads in flight.
template <bool I64>
__device__ __forceinline__ void count_slots(const ExpertSortArgs& g, int64_t s0, int64_t s1, int stride, int* count) {
  for (; s0 < s1; s0 += 8 * stride) {
    int v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = s0 + q * stride < s1 ? slot_class<I64>(g, (int)(s0 + q * stride)) : -1;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (v[q] >= 0) count_slot(count + v[q]);
  }
}

// Exclusive sums of n counts, by one wave: lane l over counts l * c .. + c.
__device__ __forceinline__ void exclusive_sums(int* v, int n, int lane) {
  const int per = (n + 63) / 64, e0 = min(lane * per, n), e1 = min(e0 + per, n);
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += v[e];
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  int at = incl - sum;
  for (int e = e0; e < e1; ++e) {
    const int c = v[e];
    v[e] = at;
    at += c;
  }
}

// The places of a wave's segment [s0, s1): next[v] is the next place of class v (kept up to date).
// FINAL: order is written too, and slots of no expert get -1; else place holds the number handed out.
template <bool I64, bool FINAL>
__device__ __forceinline__ void place_segment(const ExpertSortArgs& g, int64_t s0, int64_t s1, int bits, int* next, int lane) {
  for (; s0 < s1; s0 += 64 * 4) {  // four loads in flight
    int v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t s = s0 + 64 * q + lane;
      v[q] = s < s1 ? slot_class<I64>(g, (int)s) : -1;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint64_t same = __builtin_amdgcn_ballot_w64(v[q] >= 0);
      if (same == 0) break;
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __builtin_amdgcn_ballot_w64((v[q] >> b) & 1);
        same &= (v[q] >> b) & 1 ? set : ~set;
      }
      if (v[q] >= 0) {
        const int below = lanes_below(same), first = next[v[q]], p = first + below, s = (int)(s0 + 64 * q + lane);
        if (FINAL) {
          g.place[s] = v[q] < g.experts ? p : -1;
          g.order[p] = v[q] < g.experts ? s : -1;
        } else {
          g.place[s] = p;
        }
        // (the wave's reads above come before this write: LDS runs a wave's accesses in order)
        if (below == 0) next[v[q]] = first + __builtin_popcountll(same);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    }
  }
}

// A wave's segment of chunk `chunk` of `steps` steps a wave.
struct Segment {
  int64_t s0, s1;
};
__device__ __forceinline__ Segment segment_of(const ExpertSortArgs& g, int chunk, int wave, int steps) {
  const int64_t s0 = ((int64_t)chunk * kSortWaves + wave) * steps * 64, s1 = s0 + (int64_t)steps * 64;
  return {s0 < g.n ? s0 : g.n, s1 < g.n ? s1 : g.n};
}

template <bool I64>
__global__ __launch_bounds__(kSortThreads) void expert_sort_one(ExpertSortArgs g, int steps, int bits) {
  __shared__ SortCounts c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, classes = g.experts + 1, chunk = blockIdx.x;
  for (int e = tid; e < classes; e += kSortThreads) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c.wave[w][e] = 0;
    c.before[e] = c.all[e] = 0;
  }
  __syncthreads();
  const int64_t s0 = segment_of(g, chunk, 0, steps).s0, s1 = segment_of(g, chunk, kSortWaves - 1, steps).s1;
  const Segment seg = segment_of(g, chunk, wave, steps);
  count_slots<I64>(g, seg.s0 + lane, seg.s1, 64, c.wave[wave]);
  count_slots<I64>(g, tid, s0, kSortThreads, c.before);
  count_slots<I64>(g, s1 + tid, g.n, kSortThreads, c.all);
  __syncthreads();
  for (int e = tid; e < classes; e += kSortThreads) {
    int at = c.before[e];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = c.wave[w][e];
      c.wave[w][e] = at;
      at += n;
    }
    c.all[e] += at;
  }
  __syncthreads();
  if (wave == 0) exclusive_sums(c.all, classes, lane);
  __syncthreads();
  for (int e = tid; e < classes; e += kSortThreads) {
    const int start = c.all[e];
    if (chunk == 0) g.offsets[e] = start;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c.wave[w][e] += start;
  }
  __syncthreads();
  place_segment<I64, true>(g, seg.s0, seg.s1, bits, c.wave[wave], lane);
}

template <bool I64>
__global__ __launch_bounds__(kSortThreads) void expert_sort_count(ExpertSortArgs g, int steps, int bits) {
  __shared__ SortCounts c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, classes = g.experts + 1, chunk = blockIdx.x;
  for (int e = tid; e < classes; e += kSortThreads)
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c.wave[w][e] = 0;
  __syncthreads();
  const Segment seg = segment_of(g, chunk, wave, steps);
  count_slots<I64>(g, seg.s0 + lane, seg.s1, 64, c.wave[wave]);
  __syncthreads();
  for (int e = tid; e < classes; e += kSortThreads) {
    int at = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = c.wave[w][e];
      c.wave[w][e] = at;
      at += n;
    }
    g.counts[(int64_t)chunk * classes + e] = at;
  }
  __syncthreads();
  place_segment<I64, false>(g, seg.s0, seg.s1, bits, c.wave[wave], lane);
}

template <bool I64>
__global__ __launch_bounds__(kSortThreads) void expert_sort_place(ExpertSortArgs g, int chunks, int steps) {
  __shared__ int before[kMaxExperts + 1], all[kMaxExperts + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, classes = g.experts + 1, chunk = blockIdx.x;
  for (int e = tid; e < classes; e += kSortThreads) before[e] = all[e] = 0;
  __syncthreads();
  // column sums over the chunks: 64 classes by 8 waves at a time, 16 rows in flight
  for (int e0 = 0; e0 < classes; e0 += 64) {
    const int e = e0 + lane;
    int b = 0, a = 0;
    if (e < classes) {
      for (int q0 = wave * 16; q0 < chunks; q0 += 16 * kSortWaves) {
        int n[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) n[q] = q0 + q < chunks ? g.counts[(int64_t)(q0 + q) * classes + e] : 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (q0 + q < chunk) b += n[q];
          a += n[q];
        }
      }
      if (b != 0) __hip_atomic_fetch_add(before + e, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      if (a != 0) __hip_atomic_fetch_add(all + e, a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  }
  __syncthreads();
  if (wave == 0) exclusive_sums(all, classes, lane);
  __syncthreads();
  for (int e = tid; e < classes; e += kSortThreads) {
    if (chunk == 0) g.offsets[e] = all[e];
    before[e] += all[e];
  }
  __syncthreads();
  const int64_t s0 = segment_of(g, chunk, 0, steps).s0, s1 = segment_of(g, chunk, kSortWaves - 1, steps).s1;
  for (int64_t at = s0 + tid; at < s1; at += 4 * kSortThreads) {  // four slots in flight
    int v[4], rank[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t s = at + q * kSortThreads;
      v[q] = -1;
      if (s < s1) {
        v[q] = slot_class<I64>(g, (int)s);
        rank[q] = g.place[s];
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int s = (int)(at + q * kSortThreads);
      if (v[q] < 0) continue;
      const int p = before[v[q]] + rank[q];
      g.place[s] = v[q] < g.experts ? p : -1;
      g.order[p] = v[q] < g.experts ? s : -1;
    }
  }
}

// ------------------------------------------------------------------------------------
// Rows. A thread holds eight columns of a token: reads them once and writes them to every place of
// the token (gather), or sums the token's rows there in float32, choice by choice (combine). Bound
// by memory: 16384 tokens, 4 choices, 4096 columns (671 MB) gathered in 107 us after other work and 118 to 122
// in a loop (5.5 to 6.3 TB/s), combined in 144 and 122 to 125 (4.7 to 5.5; a token's rows lie far apart, and two
// tokens a thread are slower); 4095 x 8 x 2048 (151 MB) 27 and 29.
// The workgroups past `main` zero the rows behind the last one in use.
__device__ __forceinline__ int rows_in_use(const ExpertRowsArgs& g) {
  const int n = g.offsets[g.experts];
  return n < 0 ? 0 : n < g.rows ? n : g.rows;
}
constexpr int kRestGroups = 64;
__device__ __forceinline__ void zero_rest_rows(const ExpertRowsArgs& g, int part, uint32_t cpr) {
  const half8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  every_nth_row(rows_in_use(g) + (int64_t)part, g.rows, kRestGroups, [&](int64_t r) {
    for (uint32_t c = threadIdx.x; c < cpr; c += 256)
      store_half8(g.dst + r * g.ldd + 8 * c, zero, g.H - 8 * (int)c);
  });
}

__global__ __launch_bounds__(256) void expert_gather(ExpertRowsArgs g, uint32_t main) {
  const uint32_t cpr = ((uint32_t)g.H + 7) / 8;
  if (blockIdx.x >= main) return zero_rest_rows(g, (int)(blockIdx.x - main), cpr);
  const uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= (uint64_t)g.tokens * cpr) return;
  const uint32_t t = (uint32_t)u / cpr, c = (uint32_t)u - t * cpr;  // the host keeps the chunks below 2^32
  const int n = g.H - 8 * (int)c;
  const half8 x = load_half8(g.src + (int64_t)t * g.lds_ + 8 * c, (int)(8 * c), n);
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
        y[q] = load_half8(g.src + (int64_t)p * g.lds_ + 8 * c, (int)(8 * c), n);
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
// slots are neighbouring waves, which share dout's row in the caches): 16384 x 4 x 4096 (1.2 GB) in 223 us after
// other work and 234 to 257 in a loop, 4.7 to 5.4 TB/s.
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
      const half8 a = load_half8(d + 8 * c, (int)(8 * c), n), b = g.dweights != nullptr ? load_half8(y + 8 * c, (int)(8 * c), n) : a;
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
  int bits = 1;
  while ((g.experts >> bits) != 0) ++bits;
  const int64_t steps_in_all = ceil_div(g.n, kSortThreads);
  if (g.n <= kSortOneLaunch) {
    const unsigned chunks = g.n == 0 ? 1 : (unsigned)steps_in_all;  // one step a wave
    hipLaunchKernelGGL(expert_sort_one<I64>, dim3(chunks), dim3(kSortThreads), 0, s, g, 1, bits);
    return hipGetLastError();
  }
  // four steps a wave (2048 slots a chunk) up to kSortChunks chunks, then longer ones
  const int64_t least = ceil_div(steps_in_all, kSortChunks);
  const int steps = (int)(least < 4 ? 4 : least), chunks = (int)ceil_div(steps_in_all, steps);
  hipLaunchKernelGGL(expert_sort_count<I64>, dim3(chunks), dim3(kSortThreads), 0, s, g, steps, bits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(expert_sort_place<I64>, dim3(chunks), dim3(kSortThreads), 0, s, g, chunks, steps);
  return hipGetLastError();
}

uint32_t chunk_groups(const ExpertRowsArgs& g) { return (uint32_t)ceil_div((int64_t)g.tokens * ceil_div(g.H, 8), 256); }

}  // namespace

hipError_t launch_expert_sort(const ExpertSortArgs& g, hipStream_t s) {
  return g.ids_i64 ? launch_sort<true>(g, s) : launch_sort<false>(g, s);
}

hipError_t launch_expert_gather(const ExpertRowsArgs& g, hipStream_t s) {
  // (without slots no row goes anywhere, and src may be null: none is read)
  const uint32_t main = g.k == 0 ? 0 : chunk_groups(g), all = main + (g.offsets != nullptr ? kRestGroups : 0);
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
