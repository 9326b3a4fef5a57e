// tgemm_orth_api.cpp -- host side of the orthogonalisation (declared in include/tgemm_ops.h):
// argument validation, workspace layout and launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tgemm_ops.h"
#include "tgemm_orth.h"

namespace {

using tgemm::OrthArgs;

constexpr int64_t kMaxM = 1 << 15, kMaxSteps = 64;

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Sizes the kernels take: rows of a padded matrix in a 32-bit buffer range, tiles of a batch in
// one grid.
int check_sizes(int64_t batch, int64_t R, int64_t C) {
  if (batch < 0 || R < 0 || C < 0 || batch >= TGEMM_MAX_DIM || R >= TGEMM_MAX_DIM || C >= TGEMM_MAX_DIM)
    return TGEMM_EINVAL_DIM;
  if (batch == 0 || R == 0 || C == 0) return TGEMM_OK;
  const int64_t m = round_up(R < C ? R : C, tgemm::kOrthPad), n = round_up(R < C ? C : R, tgemm::kOrthPad);
  if (m > kMaxM || n > TGEMM_FAST_MAX_LD) return TGEMM_EINVAL_DIM;
  // Chunks of eight values of a matrix are numbered in 32 bits; the runtime takes fewer than 2^32
  // threads per launch (512 a workgroup: orth_start's groups bound the products' tiles, and the
  // norm has at most 1024 + batch workgroups).
  if (m * n / 8 >= ((int64_t)1 << 31) || batch >= ((int64_t)1 << 22)) return TGEMM_EINVAL_DIM;
  return batch * tgemm::ceil_div(m * n, 8 * 512) >= ((int64_t)1 << 23) ? TGEMM_EINVAL_DIM : TGEMM_OK;
}

// Places the workspace's arrays (each on a 256-byte boundary) from base on; returns its bytes.
int64_t place(OrthArgs& g, char* base) {
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    char* const p = base + at;
    at += round_up(bytes, 256);
    return p;
  };
  const int64_t b = g.batch, m = g.mp, x = b * m * g.np * 2;
  g.parts = reinterpret_cast<double*>(take(b * tgemm::kOrthParts * 8));
  for (int i = 0; i < 2; ++i) {
    g.hi[i] = reinterpret_cast<_Float16*>(take(x));
    g.lo[i] = reinterpret_cast<_Float16*>(take(x));
  }
  for (int i = 0; i < 2; ++i) {
    g.E[i] = reinterpret_cast<_Float16*>(take(b * m * m * 2));
    g.P[i] = reinterpret_cast<_Float16*>(take(b * m * m * 2));
  }
  g.D = reinterpret_cast<float*>(take(b * m * 4));
  g.DP = reinterpret_cast<float*>(take(b * m * 4));
  return at;
}

OrthArgs sized(int64_t batch, int64_t R, int64_t C) {
  OrthArgs g{};
  g.batch = (int)batch;
  g.R = (int)R;
  g.C = (int)C;
  g.tall = R > C;
  g.mp = (int)round_up(R < C ? R : C, tgemm::kOrthPad);
  g.np = (int)round_up(R < C ? C : R, tgemm::kOrthPad);
  // about 4096 values per workgroup of the norm, four workgroups per compute unit over the batch
  const int64_t want = tgemm::ceil_div(R * C, 4096), most = tgemm::ceil_div(1024, batch);
  const int64_t parts = want < most ? want : most;
  g.nparts = (int)(parts < 1 ? 1 : parts > tgemm::kOrthParts ? tgemm::kOrthParts : parts);
  return g;
}

}  // namespace

extern "C" {

int64_t orthogonalize_workspace_bytes(int64_t batch, int64_t R, int64_t C) {
  const int v = check_sizes(batch, R, C);
  if (v != TGEMM_OK) return v;
  if (batch == 0 || R == 0 || C == 0) return 0;
  OrthArgs g = sized(batch, R, C);
  return place(g, nullptr);
}

int orthogonalize_f16(int64_t batch, int64_t R, int64_t C, int dtype, const void* G, int64_t ldg, int64_t stride_g,
                      void* X, int64_t ldx, int64_t stride_x, int steps, float a, float b, float c, float scale,
                      void* workspace, int64_t workspace_bytes, void* stream) {
  const int v = check_sizes(batch, R, C);
  if (v != TGEMM_OK) return v;
  if (steps < 1 || steps > kMaxSteps || (dtype != TGEMM_DTYPE_F16 && dtype != TGEMM_DTYPE_F32)) return TGEMM_EINVAL_DIM;
  const int64_t cmin = C > 1 ? C : 1;
  if (ldg < cmin || ldx < cmin || stride_g < 0 || stride_x < 0) return TGEMM_EINVAL_LD;
  // results of a batch may not overlap
  if (batch > 1 && R > 0 && stride_x < (R - 1) * ldx + C) return TGEMM_EINVAL_LD;
  if (batch == 0 || R == 0 || C == 0) return TGEMM_OK;
  if (G == nullptr || X == nullptr || workspace == nullptr) return TGEMM_ENULL;
  const uintptr_t gmask = dtype == TGEMM_DTYPE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(G) & gmask) || (reinterpret_cast<uintptr_t>(X) & 1u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return TGEMM_EALIGN;
  OrthArgs g = sized(batch, R, C);
  if (workspace_bytes < place(g, static_cast<char*>(workspace))) return TGEMM_EWORKSPACE;
  int dev = -1;
  const int d = tgemm::current_device(&dev);
  if (d != TGEMM_OK) return d;
  g.G = G;
  g.X = static_cast<_Float16*>(X);
  g.ldg = ldg;
  g.stride_g = stride_g;
  g.ldx = ldx;
  g.stride_x = stride_x;
  g.f32 = dtype == TGEMM_DTYPE_F32;
  g.a = a;
  g.b = b;
  g.c = c;
  g.scale = scale;
  return tgemm::launch_orthogonalize(g, steps, static_cast<hipStream_t>(stream), dev) == hipSuccess ? TGEMM_OK
                                                                                                  : TGEMM_ELAUNCH;
}

}  // extern "C"
