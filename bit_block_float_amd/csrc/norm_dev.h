// norm_dev.h -- arguments of the layer norm kernels and their internal (hidden)
// host launchers; argument checks happen in api_norm.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hif4 {

struct NormArgs {
  const void* x;
  int64_t rows, ld;
  int c;
  bool vec;  // c % 8 == 0, and every row of x, y, weight and bias is 16-byte aligned
  const void *w, *b;
  bool w_bf16;
  float eps;
  void* y;  // plain output, of x's type
  int64_t ldy;
  float *mean, *rstd;  // either may be NULL
  uint8_t* codes;      // HiF4 [rows][c/2] or E4M3 [rows][kp]
  uint32_t* meta;      // HiF4
  const uint8_t* mask;
  uint16_t* kept;
  int n_mask;
  int kp;           // E4M3: c rounded up to 128
  uint8_t* scales;  // E4M3 [rows][lds]
  int64_t lds;
};

struct NormBackArgs {
  const void *dy, *x;
  int64_t rows, lddy, ldx, lddx;
  int c;
  bool vec;  // as above, for x, dy, dx and weight
  const void* w;
  bool w_bf16;
  const float *mean, *rstd;
  void* dx;
  float* parts;  // NULL: no weight or bias gradient
};

}  // namespace hif4

hipError_t hif4_launch_layer_norm(const hif4::NormArgs& a, bool x_bf16, int out, hipStream_t stream);
int hif4_layer_norm_backward_parts(int64_t rows, int64_t c);
hipError_t hif4_launch_layer_norm_backward(const hif4::NormBackArgs& a, bool x_bf16, void* dw,
                                           void* db, hipStream_t stream);
