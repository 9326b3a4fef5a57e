// tgemm_pingpong.h -- the two-group ping-pong schedule, for kernels that bring their own
// copies, fragment reads and MFMAs (the MXFP4 products, the orthogonalisation's products).
#pragma once

#include <type_traits>
#include <utility>

#include "tgemm_device.h"

namespace tgemm {
namespace {

// The descriptors of an operand's k-tiles, one after another: a pointer that moves by a tile (no
// 64-bit product per tile: the scalar instructions around a copy are what small tiles wait for).
struct TileStream {
  const char* p;
  int64_t step;
  uint32_t full, last;
  int left;  // tiles from this one on
  template <typename Op>
  __device__ __forceinline__ void init(const Op& op, int nk) {
    p = op.base;
    step = op.step;
    full = op.rng_full;
    last = op.rng_last;
    left = nk;
  }
  __device__ __forceinline__ bool at_last() const { return left == 1; }
  // The tile's descriptor (an empty range past the last tile, where p may lie behind the matrix).
  __device__ __forceinline__ int4v next() {
    const int4v r = make_rsrc(p, left > 1 ? full : left == 1 ? last : 0u);
    p += step;
    --left;
    return r;
  }
};

// 8 waves in two groups of four (one wave of each per SIMD) over a ring of STAGES LDS slots;
// tile t lives in slot t % STAGES. In every interval between two barriers one group issues
// MFMAs from registers while the other reads LDS and issues copies:
//   iteration kt: group 0: MFMAs of tile kt; wait for its copies of tile kt+1; barrier; reads
//                          tile kt+1; copies tile kt+STAGES (into tile kt's slot, whose last
//                          reads, group 1's, come before barrier kt);
//                 group 1: reads tile kt; copies tile kt+STAGES-1 (into tile kt-1's slot, read
//                          by both groups before barrier kt-1); wait for its copies of tile
//                          kt+1; barrier; MFMAs of tile kt.
// copy(t, group) issues at least PT0 (group 0) or PT1 (group 1) vector-memory copies of tile t
// in every call (t = 0, 1, 2, ...), also past the last tile (empty ranges), so with PT * (STAGES - 2) operations
// left in flight everything a thread copied for tile kt+1 has landed; more copies in a call
// only make that wait longer. MID adds a barrier between the phases, which measured faster
// for 256 x 256 tiles with both operands k-contiguous in the binary16 kernel.
// sched_barrier(0) pins the phases: MFMAs only touch registers, so s_barrier does not order
// them.
template <int STAGES, int PT0, int PT1, bool MID, typename Copy, typename Read, typename Mma>
__device__ __forceinline__ void pingpong_schedule(int grp, int nk, Copy&& copy, Read&& read, Mma&& mma) {
  static_assert(STAGES >= 3 && (PT0 + 2) * STAGES < 64 && PT1 <= PT0, "ring depth / vmcnt budget");
  using G0 = std::integral_constant<int, 0>;
  using G1 = std::integral_constant<int, 1>;
  if (grp == 0) {
#pragma unroll
    for (int t = 0; t < STAGES; ++t) copy(t, G0{});
    wait_vmcnt<PT0 * (STAGES - 1)>();
  } else {
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t) copy(t, G1{});
    wait_vmcnt<PT1 * (STAGES - 2)>();
  }
  lds_barrier();
  if (grp == 0) {
    read(0);
    for (int kt = 0; kt < nk; ++kt) {
      __builtin_amdgcn_sched_barrier(0);
      mma();
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<PT0 * (STAGES - 2)>();
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      read(kt + 1);  // (past the last tile: a settled slot, unused)
      copy(kt + STAGES, G0{});
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (MID) lds_barrier();
    }
  } else {
    for (int kt = 0; kt < nk; ++kt) {
      __builtin_amdgcn_sched_barrier(0);
      read(kt);
      copy(kt + STAGES - 1, G1{});
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<PT1 * (STAGES - 2)>();
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      mma();
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (MID) lds_barrier();
    }
  }
  wait_vmcnt<0>();
}

// The two wave groups of a kernel that gives each group half of every k-tile hold partial sums
// of the same wave tiles: wave w and w + 4. Each passes half of its rows of 16 x 16 tiles to the
// other through LDS (16 bytes a lane, 2 KB FM per wave, all waves at the ring's place) and adds
// what it gets to the half it keeps: group 0 rows 0 .. FM / 2 - 1, group 1 the others, in out.
// Called by every wave once the ring is free.
template <int FM, int FN, typename V>
__device__ __forceinline__ void join_k_groups(char* smem, const V (&acc)[FM][FN], V (&out)[FM / 2][FN], int wave, int lane) {
  constexpr int H = FM / 2, WAVE = H * FN * 64 * 16;
  const bool second = wave >= 4;
#pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const V give = second ? acc[i][j] : acc[i + H][j];
      out[i][j] = second ? acc[i + H][j] : acc[i][j];
      *(TG_LDS V*)(smem + wave * WAVE + ((i * FN + j) * 64 + lane) * 16) = give;
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) out[i][j] += *(const TG_LDS V*)(smem + (wave ^ 4) * WAVE + ((i * FN + j) * 64 + lane) * 16);
  __syncthreads();
}

// Stores a staged tile (StagedTile) to any C: 16-byte chunks where `vec` says that every
// chunk of C is 16-byte aligned, single elements otherwise and in a chunk that N cuts. NT: the
// result streams out (store_c); false for one that the next kernel reads.
template <typename ST, int WTM, bool NT = true>
__device__ __forceinline__ void store_staged(const char* region, int lane, _Float16* C, int64_t ldc, int mvalid,
                                             int nvalid, int vec) {
#pragma unroll
  for (int i = 0; i < WTM * ST::SCPR / 64; ++i) {
    const int idx = i * 64 + lane;
    const int r = idx / ST::SCPR, c = idx % ST::SCPR;
    if (c >= ST::CPR) continue;
    const half8 x = *(const TG_LDS half8*)(region + r * ST::RB + (ST::chunk_at(r, c) << 4));
    if (r >= mvalid || 8 * c >= nvalid) continue;
    _Float16* const p = C + (int64_t)r * ldc + 8 * c;
    if (vec && 8 * c + 8 <= nvalid) {
      if (NT)
        store_c(p, x);
      else
        *(half8*)p = x;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * c + e < nvalid) p[e] = x[e];
    }
  }
}

}  // namespace
}  // namespace tgemm
