// Calls an entry point of the expert layer or the norm with the host code of its kernels' file linked
// in, and the HIP runtime replaced by one that records launches: no GPU, no HIP runtime library. Prints
// a line per launch, the kernel, its workgroups, and the count of `main` workgroups that the expert layer's
// kernels take as their second argument, then the return code.
//   driver gather TOKENS K ROWS H X PLACE XS OFFSETS EXPERTS      (pointers as numbers; never read)
//   driver norm ROWS K RESIDUAL_DTYPE(-1: none) Y Q
//   driver rows FIRST ROWS N          (no entry point: the rows that a zeroing workgroup goes over, one a line)
//   driver k_tiles K BK               (no entry point: the k-tiles of a product, and k values in the last)
//   driver combine_grad TOKENS K ROWS H DOUT Y PLACE DY OFFSETS EXPERTS
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

#include "tgemm_expert.h"
#include "tgemm_ops.h"

namespace {
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> k;
  return k;
}
struct {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
} pushed;
int64_t number(const char* s) { return std::strtoll(s, nullptr, 0); }
void* pointer(const char* s) { return reinterpret_cast<void*>((uintptr_t)number(s)); }
}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  kernels()[host] = name;
}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  pushed = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *lds = pushed.lds;
  *stream = pushed.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3, void** args, size_t, hipStream_t) {
  const std::string& name = kernels()[f];
  const bool of_rows = name.find("expert_") != std::string::npos;
  std::printf("%s %u %u\n", name.c_str(), grid.x, of_rows ? *static_cast<const uint32_t*>(args[1]) : 0u);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}

namespace tgemm {
int current_device(int* device) {
  *device = 0;
  return TGEMM_OK;
}
hipError_t launch_expert_gemm(int, ExpertForm, const ExpertGemmArgs&, hipStream_t, int) { return hipErrorNotSupported; }
}  // namespace tgemm

int main(int argc, char** argv) {
  int rc = 0;
  if (argc == 11 && !std::strcmp(argv[1], "gather")) {
    const int64_t H = number(argv[5]), ld = H > 1 ? H : 1;
    rc = expert_gather_f16(number(argv[2]), number(argv[3]), number(argv[4]), H, pointer(argv[6]), ld, pointer(argv[7]),
                           pointer(argv[8]), ld, pointer(argv[9]), number(argv[10]), nullptr);
  } else if (argc == 12 && !std::strcmp(argv[1], "combine_grad")) {
    const int64_t H = number(argv[5]), ld = H > 1 ? H : 1;
    rc = expert_combine_f16_backward(number(argv[2]), number(argv[3]), number(argv[4]), H, pointer(argv[6]), ld, pointer(argv[7]),
                                     ld, pointer(argv[8]), nullptr, TGEMM_DTYPE_F32, pointer(argv[9]), ld, nullptr,
                                     pointer(argv[10]), number(argv[11]), nullptr);
  } else if (argc == 7 && !std::strcmp(argv[1], "norm")) {
    const int64_t K = number(argv[3]);
    const int dtype = (int)number(argv[4]);
    void* const some = reinterpret_cast<void*>(256);
    void* const residual = dtype < 0 ? nullptr : some;
    void* const q = pointer(argv[6]);
    rc = rmsnorm_f16(number(argv[2]), K, some, K, residual, K, dtype, some, TGEMM_DTYPE_F16, 1e-6f, residual, K, pointer(argv[5]), K,
                     q, K, static_cast<float*>(q), nullptr);
  } else if (argc == 5 && !std::strcmp(argv[1], "rows")) {
    tgemm::every_nth_row(number(argv[2]), number(argv[3]), number(argv[4]), [](int64_t r) { std::printf("row %lld 0\n", (long long)r); });
  } else if (argc == 4 && !std::strcmp(argv[1], "k_tiles")) {
    const int K = (int)number(argv[2]), BK = (int)number(argv[3]), nk = tgemm::k_tiles(K, BK);
    std::printf("k_tiles %d %d\n", nk, nk > 0 ? K - (nk - 1) * BK : 0);
  } else {
    return 2;
  }
  std::printf("rc %d\n", rc);
  return 0;
}
