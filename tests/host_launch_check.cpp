// host_launch_check.cpp -- the host code of the 8-bit linear layers and the
// layer norm (csrc/api_fp8.hip, fp8.hip, gemm_fp8.hip, api_norm.hip, norm.hip),
// run without a GPU under AddressSanitizer and UndefinedBehaviorSanitizer.
//
// The few HIP functions that this code calls are defined here: there is one
// gfx950 device, a launch is recorded and not run. So the size queries, the
// choice of a kernel and its grid are walked over sizes around each of their
// borders, up to the largest that the entry points take.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>
#include <vector>

#include "hif4.h"

static int failures = 0;
static int launches = 0;

static void fail(const char* what, long long a, long long b, long long c) {
  fprintf(stderr, "FAIL %s (%lld, %lld, %lld)\n", what, a, b, c);
  if (++failures > 20) exit(1);
}

// ---- the HIP functions

struct Config {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
};
static std::vector<Config> configs;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*,
                           void*, int*) {}
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
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  ++launches;
  const uint64_t threads = (uint64_t)block.x * block.y * block.z;
  if (grid.x == 0 || grid.y == 0 || grid.z != 1 || threads == 0 || threads > 1024 ||
      (uint64_t)grid.x * block.x >= (1ull << 32) || (uint64_t)grid.y * block.y >= (1ull << 32))
    fail("a launch with the grid", grid.x, grid.y, block.x);
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

// ---- the walks

static char* const A = reinterpret_cast<char*>(0x100000);  // never dereferenced
static uint8_t* const U8 = reinterpret_cast<uint8_t*>(A);

static std::vector<int64_t> around(std::initializer_list<int64_t> borders) {
  std::vector<int64_t> v;
  for (int64_t b : borders)
    for (int64_t d = -1; d <= 1; ++d) v.push_back(b + d);
  return v;
}

// A product's size query and the call: a refused size needs 0 bytes, and a call
// that is given what the query says is launched.
static void linear_sizes() {
  const auto rows = around({1, 16, 17, 64, 65, 128, 129, 256, 1024, 2048, 5120, 57600, 1 << 20, (1 << 26) - 16, 1 << 26,
                            (int64_t)1 << 31});
  const auto ks = around({0, 1, 64, 128, 256, 2048, 4096, 5120, 8192, 13824, 1 << 22});
  for (int64_t m : rows)
    for (int64_t n : rows)
      for (int64_t k : ks) {
        const size_t need = hif4_linear_fp8_workspace_bytes(m, n, k);
        if ((m < 0 || n < 0 || k < 0 || k % 128 != 0) && need != 0) fail("bytes for a refused size", m, n, k);
        for (int f32 = 0; f32 < 2; ++f32) {
          const int64_t lds = k > 0 ? (k / 128 + 3) / 4 * 4 : 4;
          const int before = launches;
          const hif4_status st = hif4_linear_fp8(
              U8, U8, lds, U8, A, lds, f32 ? HIF4_SCALE_F32 : HIF4_SCALE_E8M0, 128, m, n, k, A,
              f32 ? HIF4_F32 : HIF4_BF16, A, need, nullptr);
          if (st == HIF4_OK ? m > 0 && n > 0 && k > 0 && launches == before : launches != before)
            fail("launches of a product", m, n, k);
          if (st != HIF4_OK && st != HIF4_ERR_SHAPE) fail("status of a product", m, n, k);
          if (st == HIF4_ERR_SHAPE && need != 0) fail("bytes for a refused product", m, n, k);
        }
      }
}

static void linear_backward_sizes() {
  const auto sizes = around({1, 17, 64, 128, 129, 1024, 2048, 8192, 1 << 18, 1 << 22});
  auto ks = sizes;
  for (int64_t k : around({(int64_t)1 << 30, ((int64_t)1 << 31) - 128, (int64_t)1 << 31})) ks.push_back(k);
  for (int64_t m : sizes)
    for (int64_t n : sizes)
      for (int64_t k : ks) {
        const size_t need = hif4_linear_fp8_backward_workspace_bytes(m, n, k);
        const int64_t big = 1 << 17;
        const hif4_status st = hif4_linear_fp8_backward(
            A, HIF4_BF16, n < 1 ? 1 : n, U8, U8, big, U8, A, big, HIF4_SCALE_E8M0, 128, m, n, k, A,
            HIF4_BF16, A, HIF4_F32, A, need, nullptr);
        if (st != HIF4_OK && st != HIF4_ERR_SHAPE) fail("status of a backward", m, n, k);
        if (st == HIF4_ERR_SHAPE && need != 0) fail("bytes for a refused backward", m, n, k);
        if (st == HIF4_OK && m > 0 && n > 0 && k > 0 && need == 0) fail("no bytes for a backward", m, n, k);
      }
}

static void quantize_sizes() {
  const auto rows = around({1, 128, 129, 57600, 1 << 22, 1 << 30, ((int64_t)1 << 31) - 127, (int64_t)1 << 31});
  const auto ks = around({1, 8, 128, 129, 5120, 65536, 1 << 22});
  const int64_t lds = 1 << 25;
  for (int64_t r : rows)
    for (int64_t k : ks)
      for (int dt = 0; dt < 2; ++dt)
        for (int64_t br : {1, 128}) {
          hif4_status st[4] = {
              hif4_quantize_fp8(A, dt, r, k, k < 1 ? 1 : k, br, 0, U8, U8, lds, nullptr),
              hif4_quantize_fp8(A, dt, r, k, k < 1 ? 1 : k, br, 1, U8, U8, lds, nullptr),
              hif4_quantize_fp8_both(A, dt, r, k, k < 1 ? 1 : k, br, U8, U8, lds, U8, U8, lds, nullptr),
              hif4_dequantize_fp8(U8, A, HIF4_SCALE_E8M0, br, lds, r, k, A, dt, nullptr)};
          const bool ok = r >= 0 && k >= 0 && r < (int64_t)1 << 31 && k <= 1 << 22;
          const bool many = ok && (r + 127) / 128 * ((k + 127) / 128) >= (int64_t)1 << 31;
          for (int i = 0; i < 4; ++i)
            if (st[i] != (ok && !(many && i < 3) ? HIF4_OK : HIF4_ERR_SHAPE)) fail("status of a quantizer", r, k, i);
        }
}

static void norm_sizes() {
  const auto rows = around({1, 16, 64, 512, 2048, 57600, 1 << 24, (int64_t)1 << 31});
  const auto cs = around({1, 8, 128, 256, 512, 1024, 4096, 5120, 6144, 8192, 16384, 32768, 65536});
  for (int64_t r : rows)
    for (int64_t c : cs)
      for (int dt = 0; dt < 2; ++dt) {
        const bool ok = r >= 0 && r < (int64_t)1 << 31 && c >= 1 && c <= 65536;
        const hif4_status want = ok ? HIF4_OK : HIF4_ERR_SHAPE;
        const size_t need = hif4_layer_norm_backward_workspace_bytes(r, c);
        if ((need != 0) != ok) fail("bytes of a norm's backward", r, c, dt);
        float* const f = reinterpret_cast<float*>(A);
        if (hif4_layer_norm(A, dt, r, c, c, A, A, 0, 1e-6, A, c, f, f, nullptr) != want)
          fail("status of a norm", r, c, dt);
        if (hif4_layer_norm_quantize_fp8(A, dt, r, c, c, A, A, 0, 1e-6, U8, U8, 512, nullptr) != want)
          fail("status of a norm to E4M3", r, c, dt);
        if (c % 64 == 0 && hif4_layer_norm_quantize(A, dt, r, c, c, A, A, 0, 1e-6, nullptr, 0, nullptr,
                                                    U8, (uint32_t*)A, nullptr) != want)
          fail("status of a norm to HiF4", r, c, dt);
        if (hif4_layer_norm_backward(A, c, A, c, dt, r, c, f, f, A, 0, A, c, A, A, A, need, nullptr) != want)
          fail("status of a norm's backward", r, c, dt);
      }
}

int main() {
  linear_sizes();
  linear_backward_sizes();
  quantize_sizes();
  norm_sizes();
  printf("%d launches\n", launches);
  if (failures) return 1;
  printf("host-launch-check OK\n");
  return 0;
}
