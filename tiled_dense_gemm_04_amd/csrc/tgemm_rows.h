// tgemm_rows.h -- eight consecutive values of a row, of any alignment, cut by the row's end: the
// access of the kernels that go over rows once (the norm, the rows sorted by expert). gfx950 serves
// 16-byte accesses at any address, so a whole chunk is one access whatever the strides.
#pragma once

#include "tgemm_device.h"

namespace tgemm {
namespace {

typedef unsigned int uint2v __attribute__((ext_vector_type(2)));

// The words of v (32 bits each) moved down by `elements` of BITS bits, zeros coming in.
template <int BITS, int N>
__device__ __forceinline__ void move_down(uint32_t (&v)[N], int elements) {
  const int bits = elements * BITS;
  if (N > 4 && (bits & 128)) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i + 4 < N ? v[i + 4] : 0u;
  }
  if (N > 2 && (bits & 64)) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i + 2 < N ? v[i + 2] : 0u;
  }
  if (bits & 32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i + 1 < N ? v[i + 1] : 0u;
  }
  if (bits & 16) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_alignbit(i + 1 < N ? v[i + 1] : 0u, v[i], 16);
  }
}

// p: the chunk's first element; at: elements of the row before it (0, or 8 or more); n: elements from there
// to the row's end (n <= 0: none; p may then lie outside the matrix and is not used). Elements past the
// end are zero, and never written. The last chunk of a row is loaded as the row's last eight elements,
// in one access, and moved into place: element by element, each load waits for the one before (norm of 16384 x
// 4095 with a binary16 residual 161 us, so 115; its gradient 142 and 96; 4096 columns 98 and 84).
template <typename T, int BITS>
__device__ __forceinline__ void load_chunk(const T* p, int at, int n, uint32_t (&v)[BITS / 4]) {
  constexpr int N = BITS / 4;  // words of eight elements
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0u;
  if (n >= 8 || (n > 0 && at >= 8)) {
    const int past = n >= 8 ? 0 : 8 - n;
    __builtin_memcpy(v, p - past, BITS);
    if (past > 0) move_down<BITS>(v, past);
  } else if (n > 0) {  // a row of fewer than eight
    T row[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) row[e] = p[e];
    __builtin_memcpy(v, row, BITS);
  }
}
__device__ __forceinline__ half8 load_half8(const _Float16* p, int at, int n) {
  uint32_t v[4];
  load_chunk<_Float16, 16>(p, at, n, v);
  half8 h;
  __builtin_memcpy(&h, v, 16);
  return h;
}
__device__ __forceinline__ void load_float8(const float* p, int at, int n, float (&f)[8]) {
  uint32_t v[8];
  load_chunk<float, 32>(p, at, n, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i]);
}
// Eight elements of v to p, or the first n: four, two and one.
template <typename T, int BITS>
__device__ __forceinline__ void store_chunk(T* p, uint32_t (&v)[BITS / 4], int n) {
  if (n >= 8) {
    __builtin_memcpy(p, v, BITS);
  } else if (n > 0) {
    if (n & 4) {
      __builtin_memcpy(p, v, BITS / 2);
      p += 4;
      move_down<BITS>(v, 4);
    }
    if (n & 2) {
      __builtin_memcpy(p, v, BITS / 4);
      p += 2;
      move_down<BITS>(v, 2);
    }
    if (n & 1) __builtin_memcpy(p, v, BITS / 8);
  }
}
__device__ __forceinline__ void store_half8(_Float16* p, const half8& h, int n) {
  uint32_t v[4];
  __builtin_memcpy(v, &h, 16);
  store_chunk<_Float16, 16>(p, v, n);
}
__device__ __forceinline__ void store_float8(float* p, const float (&f)[8], int n) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(f[i]);
  store_chunk<float, 32>(p, v, n);
}
__device__ __forceinline__ void store_bytes8(uint8_t* p, const uint2v& b, int n) {
  uint32_t v[2] = {b[0], b[1]};
  store_chunk<uint8_t, 8>(p, v, n);
}

}  // namespace
}  // namespace tgemm
