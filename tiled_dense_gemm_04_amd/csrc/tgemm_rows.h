// tgemm_rows.h -- eight consecutive values of a row, of any alignment, cut by the row's end: the
// access of the kernels that go over rows once (the norm, the rows sorted by expert). gfx950 serves
// 16-byte accesses at any address, so a whole chunk is one access whatever the strides.
#pragma once

#include "tgemm_device.h"

namespace tgemm {
namespace {

typedef unsigned int uint2v __attribute__((ext_vector_type(2)));

// p: the chunk's first element; n: elements from there to the row's end (n <= 0: none; p may then
// lie outside the matrix and is not used). Elements past the end are zero, and never written.
__device__ __forceinline__ half8 load_half8(const _Float16* p, int n) {
  half8 v = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n >= 8) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) v[e] = p[e];
  }
  return v;
}
__device__ __forceinline__ void load_float8(const float* p, int n, float (&v)[8]) {
  if (n >= 8) {
    __builtin_memcpy(v, p, 32);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.0f;
  }
}
__device__ __forceinline__ void store_half8(_Float16* p, const half8& v, int n) {
  if (n >= 8) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void store_float8(float* p, const float (&v)[8], int n) {
  if (n >= 8) {
    __builtin_memcpy(p, v, 32);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) p[e] = v[e];
  }
}
__device__ __forceinline__ void store_bytes8(uint8_t* p, const uint2v& v, int n) {
  if (n >= 8) {
    __builtin_memcpy(p, &v, 8);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < n) p[e] = (uint8_t)(v[e / 4] >> (8 * (e % 4)));
  }
}

}  // namespace
}  // namespace tgemm
