// mxfp4_launch_check.cpp -- the host code of the 4-bit microscaled layers (csrc/
// api_mxfp4.hip, mxfp4.hip, gemm_mxfp4.hip), run without a GPU under AddressSanitizer
// and UndefinedBehaviorSanitizer.
//
// The few HIP functions that this code calls are defined here: there is one gfx950
// device, a launch is recorded and not run. So the size queries, the choice of a kernel
// and its grid are walked over sizes around each of their borders, up to the largest
// that the entry points take.
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
static const int64_t* const I64 = reinterpret_cast<const int64_t*>(A);

static std::vector<int64_t> around(std::initializer_list<int64_t> borders) {
  std::vector<int64_t> v;
  for (int64_t b : borders)
    for (int64_t d = -1; d <= 1; ++d) v.push_back(b + d);
  return v;
}

static void linear() {
  const auto rows = around({1, 16, 17, 32, 64, 128, 129, 256, 1024, 4096, 5120, 57600, 1 << 20, 1 << 26, (int64_t)1 << 31});
  const auto ks = around({0, 64, 128, 256, 384, 1024, 4096, 8192, 13824, 1 << 22});
  for (int64_t m : rows)
    for (int64_t n : rows)
      for (int64_t k : ks) {
        const size_t need = hif4_linear_mxfp4_workspace_bytes(m, n, k);
        if ((m < 0 || n < 0 || k < 0 || k % 128 != 0) && need != 0) fail("bytes for a refused size", m, n, k);
        const int before = launches;
        const hif4_status st = hif4_linear_mxfp4(U8, U8, U8, U8, m, n, k, A, HIF4_BF16, A, need, nullptr);
        if (st == HIF4_OK ? m > 0 && n > 0 && k > 0 && launches == before : launches != before)
          fail("launches of a product", m, n, k);
        if (st != HIF4_OK && st != HIF4_ERR_SHAPE) fail("status of a product", m, n, k);
        if (st == HIF4_ERR_SHAPE && need != 0) fail("bytes for a refused product", m, n, k);
      }
}

static void grouped() {
  const auto rows = around({1, 6, 16, 128, 1024, 57600, 1 << 22, (int64_t)1 << 31});
  const auto ns = around({1, 16, 64, 128, 5120, 1 << 15, 1 << 24});
  for (int64_t m : rows)
    for (int64_t n : ns)
      for (int64_t g : around({1, 2, 64, 1024, 1 << 16}))
        for (int64_t k : {(int64_t)0, (int64_t)128, (int64_t)2048, (int64_t)5120, (int64_t)1 << 22}) {
          const int before = launches;
          const hif4_status st = hif4_linear_mxfp4_grouped(U8, U8, U8, U8, I64, g, m, n, k, A, HIF4_F32, nullptr);
          const bool some = m > 0 && n > 0 && g > 0;
          if (st == HIF4_OK ? some && launches == before : launches != before) fail("launches by groups", m, n, g);
          if (st != HIF4_OK && st != HIF4_ERR_SHAPE) fail("status by groups", m, n, g);
          if (m >= 0 && m <= 57601 && n >= 0 && n <= 5121 && g >= 0 && g <= 1025 && st != HIF4_OK)
            fail("an ordinary size refused", m, n, g);
        }
}

static void backward() {
  const auto sizes = around({1, 17, 64, 129, 1024, 2048, 8192, 1 << 18, 1 << 22});
  auto ks = sizes;
  for (int64_t k : around({(int64_t)1 << 30, (int64_t)1 << 31})) ks.push_back(k);
  for (int64_t m : sizes)
    for (int64_t n : sizes)
      for (int64_t k : ks)
        for (int64_t g : {-1, 0, 1, 3, 64, 1 << 16}) {  // 0: one weight
          const int64_t ld = n < 1 ? 1 : n;
          const size_t need = g == 0 ? hif4_linear_mxfp4_backward_workspace_bytes(m, n, k)
                                     : hif4_linear_mxfp4_grouped_backward_workspace_bytes(g, m, n, k);
          const hif4_status st =
              g == 0 ? hif4_linear_mxfp4_backward(A, HIF4_BF16, ld, U8, U8, U8, U8, m, n, k, A, HIF4_BF16, A,
                                                  HIF4_F32, A, need, nullptr)
                     : hif4_linear_mxfp4_grouped_backward(A, HIF4_BF16, ld, U8, U8, U8, U8, I64, g, m, n, k, A,
                                                          HIF4_BF16, A, HIF4_F32, A, need, nullptr);
          if (st != HIF4_OK && st != HIF4_ERR_SHAPE) fail("status of a backward", m, n, k);
          if (st == HIF4_ERR_SHAPE && need != 0) fail("bytes for a refused backward", m, n, k);
          if (st == HIF4_OK && m > 0 && n > 0 && k > 0 && need == 0) fail("no bytes for a backward", m, n, k);
          if (m > 0 && m <= 8193 && n > 0 && n <= 8193 && k > 0 && k <= 8193 && g >= 0 && g <= 64 && st != HIF4_OK)
            fail("an ordinary backward refused", m, n, g);
        }
}

static void quantize() {
  const auto rows = around({1, 128, 129, 57600, 1 << 22, 1 << 30, ((int64_t)1 << 31) - 127, (int64_t)1 << 31});
  const auto ks = around({1, 8, 128, 129, 5120, 65536, 1 << 22});
  for (int64_t r : rows)
    for (int64_t k : ks)
      for (int64_t batch : {(int64_t)0, (int64_t)1, (int64_t)3, (int64_t)40000, (int64_t)1 << 31})
        for (int dt = 0; dt < 2; ++dt) {
          const int64_t ld = k < 1 ? 1 : k;
          const bool ok = r >= 0 && k >= 0 && r < (int64_t)1 << 31 && k <= 1 << 22 && batch < (int64_t)1 << 31 &&
                          batch * r < (int64_t)1 << 31;
          const hif4_status want = ok ? HIF4_OK : HIF4_ERR_SHAPE;
          if (hif4_quantize_mxfp4(A, dt, batch, r, k, ld, 0, nullptr, 0, U8, U8, nullptr) != want ||
              hif4_quantize_mxfp4(A, dt, batch, r, k, ld, 1, nullptr, 0, U8, U8, nullptr) != want ||
              hif4_quantize_mxfp4_both(A, dt, batch, r, k, ld, nullptr, 0, U8, U8, U8, U8, nullptr) != want)
            fail("status of a quantizer", r, k, batch);
          if (batch != 1) continue;
          for (int64_t g : {1, 5, 1 << 16}) {
            const int64_t cols = hif4_mxfp4_columns(r, g);
            const hif4_status w = ok && cols < (int64_t)1 << 31 ? HIF4_OK : HIF4_ERR_SHAPE;
            if (ok && (cols % 128 != 0 || cols < r || cols > r + 127 * g)) fail("columns", r, g, cols);
            if (hif4_quantize_mxfp4(A, dt, 1, r, k, ld, 1, I64, g, U8, U8, nullptr) != w) fail("quantized by groups", r, k, g);
          }
          if (hif4_dequantize_mxfp4(U8, U8, r, k, A, dt, nullptr) !=
              (r >= 0 && k >= 0 && r < (int64_t)1 << 31 ? HIF4_OK : HIF4_ERR_SHAPE))
            fail("status of the decoder", r, k, dt);
        }
}

int main() {
  linear();
  grouped();
  backward();
  quantize();
  printf("%d launches\n", launches);
  if (failures) return 1;
  printf("mxfp4-launch-check OK\n");
  return 0;
}
