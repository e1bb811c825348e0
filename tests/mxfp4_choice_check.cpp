// mxfp4_choice_check.cpp -- which kernels the products of the 4-bit microscaled layers
// launch at given sizes, without a GPU: the HIP functions that the host code calls are
// defined here, and a launch prints the kernel's name and grid instead of running.
//
// Reads calls from stdin, one a line:
//   linear m n k
//   grouped groups m n k
//   backward m n k which            which: 1 dX, 2 dW, 3 both
//   grouped_backward groups m n k which
// and prints a line for each: its status, then mangled name, grid x and grid y of every
// launch.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <map>
#include <string>
#include <vector>

#include "hif4.h"

struct Config {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
};
static std::vector<Config> configs;

// (registered by the sources' constructors, before this file's own objects exist)
static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*,
                           void*, int*) {
  names()[f] = name;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  configs.push_back({grid, block, shared, stream});
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = configs.back().grid;
  *block = configs.back().block;
  *shared = configs.back().shared;
  *stream = configs.back().stream;
  configs.pop_back();
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3, void**, size_t, hipStream_t) {
  printf(" %s %u %u", names()[f].c_str(), grid.x, grid.y);
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  memset(p, 0, sizeof(*p));
  strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
}

hipError_t hif4_launch_zero(void*, size_t, hipStream_t) { return hipSuccess; }

int main() {
  char* const A = reinterpret_cast<char*>(0x100000);  // never dereferenced
  uint8_t* const u = reinterpret_cast<uint8_t*>(A);
  const int64_t* const off = reinterpret_cast<const int64_t*>(A);
  char op[32], line[256];
  while (fgets(line, sizeof line, stdin)) {
    long long v[5] = {0, 0, 0, 0, 0};
    if (sscanf(line, "%31s %lld %lld %lld %lld %lld", op, v, v + 1, v + 2, v + 3, v + 4) < 4) return 2;
    printf("%s", op);
    int st;
    if (!strcmp(op, "linear")) {
      st = hif4_linear_mxfp4(u, u, u, u, v[0], v[1], v[2], A, HIF4_BF16, A,
                             hif4_linear_mxfp4_workspace_bytes(v[0], v[1], v[2]), nullptr);
    } else if (!strcmp(op, "grouped")) {
      st = hif4_linear_mxfp4_grouped(u, u, u, u, off, v[0], v[1], v[2], v[3], A, HIF4_BF16, nullptr);
    } else if (!strcmp(op, "backward")) {
      st = hif4_linear_mxfp4_backward(A, HIF4_BF16, v[1], u, u, u, u, v[0], v[1], v[2], v[3] & 1 ? A : nullptr,
                                      HIF4_BF16, v[3] & 2 ? A : nullptr, HIF4_F32, A,
                                      hif4_linear_mxfp4_backward_workspace_bytes(v[0], v[1], v[2]), nullptr);
    } else if (!strcmp(op, "grouped_backward")) {
      st = hif4_linear_mxfp4_grouped_backward(
          A, HIF4_BF16, v[2], u, u, u, u, off, v[0], v[1], v[2], v[3], v[4] & 1 ? A : nullptr, HIF4_BF16,
          v[4] & 2 ? A : nullptr, HIF4_F32, A,
          hif4_linear_mxfp4_grouped_backward_workspace_bytes(v[0], v[1], v[2], v[3]), nullptr);
    } else {
      return 2;
    }
    printf(" status %d\n", st);
  }
  return 0;
}
