// api_norm.hip -- the C ABI of the layer norm, declared and documented in
// include/hif4.h. Every argument check runs before any HIP call.
#include <float.h>
#include <math.h>

#include "api_util.h"
#include "norm_dev.h"

namespace {

constexpr int64_t kMaxC = 65536;

size_t elem(int dtype) { return dtype == HIF4_BF16 ? 2 : 4; }

// 16-byte rows: what lets a kernel take whole runs of 8.
bool vec_rows(const void* p, int64_t ld, int dtype) {
  return aligned(p, 16) && (ld * (int64_t)elem(dtype)) % 16 == 0;
}

hif4_status check_common(int64_t rows, int64_t c, int x_dtype, int w_dtype) {
  if (rows < 0 || rows >= (int64_t(1) << 31) || c < 1 || c > kMaxC) return HIF4_ERR_SHAPE;
  if (x_dtype != HIF4_F32 && x_dtype != HIF4_BF16) return HIF4_ERR_DTYPE;
  if (w_dtype != HIF4_F32 && w_dtype != HIF4_BF16) return HIF4_ERR_DTYPE;
  return HIF4_OK;
}

hif4_status check_forward(const void* x, int x_dtype, int64_t rows, int64_t c, int64_t ld,
                          const void* weight, const void* bias, int w_dtype, double eps,
                          hif4::NormArgs& a) {
  const hif4_status st = check_common(rows, c, x_dtype, w_dtype);
  if (st != HIF4_OK) return st;
  if (ld < c) return HIF4_ERR_SHAPE;
  if (!(eps >= 0.0 && eps <= FLT_MAX)) return HIF4_ERR_ARG;
  if (rows == 0) return HIF4_OK;
  if (!x) return HIF4_ERR_NULL;
  if (!aligned(x, elem(x_dtype)) || !aligned(weight, elem(w_dtype)) ||
      !aligned(bias, elem(w_dtype)))
    return HIF4_ERR_ALIGN;
  a = hif4::NormArgs{};
  a.x = x;
  a.rows = rows;
  a.ld = ld;
  a.c = (int)c;
  a.vec = c % 8 == 0 && vec_rows(x, ld, x_dtype) && aligned(weight, 16) && aligned(bias, 16);
  a.w = weight;
  a.b = bias;
  a.w_bf16 = w_dtype == HIF4_BF16;
  // a positive eps stays positive: a row of equal values has rstd = eps^(-1/2), not infinity
  a.eps = eps > 0.0 ? fmaxf((float)eps, FLT_TRUE_MIN) : 0.0f;
  return HIF4_OK;
}

}  // namespace

extern "C" {

hif4_status hif4_layer_norm(const void* x, int x_dtype, int64_t rows, int64_t c, int64_t ld,
                            const void* weight, const void* bias, int w_dtype, double eps, void* y,
                            int64_t ldy, float* mean, float* rstd, hipStream_t stream) {
  hif4::NormArgs a;
  hif4_status st = check_forward(x, x_dtype, rows, c, ld, weight, bias, w_dtype, eps, a);
  if (st != HIF4_OK) return st;
  if (ldy < c) return HIF4_ERR_SHAPE;
  if (rows == 0) return HIF4_OK;
  if (!y) return HIF4_ERR_NULL;
  if (!aligned(y, elem(x_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4)) return HIF4_ERR_ALIGN;
  a.y = y;
  a.ldy = ldy;
  a.vec = a.vec && vec_rows(y, ldy, x_dtype);
  a.mean = mean;
  a.rstd = rstd;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_layer_norm(a, x_dtype == HIF4_BF16, 0, stream));
}

hif4_status hif4_layer_norm_quantize(const void* x, int x_dtype, int64_t rows, int64_t c,
                                     int64_t ld, const void* weight, const void* bias, int w_dtype,
                                     double eps, const uint8_t* mask, int64_t n_mask, void* kept,
                                     uint8_t* codes, uint32_t* meta, hipStream_t stream) {
  hif4::NormArgs a;
  hif4_status st = check_forward(x, x_dtype, rows, c, ld, weight, bias, w_dtype, eps, a);
  if (st != HIF4_OK) return st;
  if (c % 64 != 0 || n_mask < 0 || (mask && n_mask > c)) return HIF4_ERR_SHAPE;
  if (rows == 0) return HIF4_OK;
  if (!codes || !meta || (mask && n_mask > 0 && !kept)) return HIF4_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(meta, 4) || !aligned(mask, 16) || !aligned(kept, 2))
    return HIF4_ERR_ALIGN;
  a.mask = mask;
  a.n_mask = mask ? (int)n_mask : 0;
  a.kept = (uint16_t*)kept;
  a.codes = codes;
  a.meta = meta;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_layer_norm(a, x_dtype == HIF4_BF16, 1, stream));
}

hif4_status hif4_layer_norm_quantize_fp8(const void* x, int x_dtype, int64_t rows, int64_t c,
                                         int64_t ld, const void* weight, const void* bias,
                                         int w_dtype, double eps, uint8_t* codes, uint8_t* scales,
                                         int64_t lds, hipStream_t stream) {
  hif4::NormArgs a;
  hif4_status st = check_forward(x, x_dtype, rows, c, ld, weight, bias, w_dtype, eps, a);
  if (st != HIF4_OK) return st;
  if (lds < (c + 127) / 128) return HIF4_ERR_SHAPE;
  if (rows == 0) return HIF4_OK;
  if (!codes || !scales) return HIF4_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(scales, 4) || lds % 4 != 0) return HIF4_ERR_ALIGN;
  a.codes = codes;
  a.scales = scales;
  a.lds = lds;
  a.kp = (int)((c + 127) / 128 * 128);
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_layer_norm(a, x_dtype == HIF4_BF16, 2, stream));
}

size_t hif4_layer_norm_backward_workspace_bytes(int64_t rows, int64_t c) {
  if (rows < 0 || rows >= (int64_t(1) << 31) || c < 1 || c > kMaxC) return 0;
  return align256((size_t)hif4_layer_norm_backward_parts(rows, c) * 2 * (size_t)c * sizeof(float));
}

hif4_status hif4_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                     int x_dtype, int64_t rows, int64_t c, const float* mean,
                                     const float* rstd, const void* weight, int w_dtype, void* dx,
                                     int64_t lddx, void* dweight, void* dbias, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  hif4_status st = check_common(rows, c, x_dtype, w_dtype);
  if (st != HIF4_OK) return st;
  if (lddy < c || ldx < c || lddx < c) return HIF4_ERR_SHAPE;
  const bool sums = dweight || dbias;
  if (rows == 0 && !sums) return HIF4_OK;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return HIF4_ERR_NULL;
  const size_t e = elem(x_dtype), we = elem(w_dtype);
  if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(weight, we) || !aligned(dweight, we) || !aligned(dbias, we))
    return HIF4_ERR_ALIGN;
  if (sums) {
    if (!workspace || workspace_bytes < hif4_layer_norm_backward_workspace_bytes(rows, c))
      return HIF4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HIF4_ERR_ALIGN;
  }
  hif4::NormBackArgs a{};
  a.dy = dy;
  a.x = x;
  a.rows = rows;
  a.lddy = lddy;
  a.ldx = ldx;
  a.lddx = lddx;
  a.c = (int)c;
  a.vec = c % 8 == 0 && vec_rows(dy, lddy, x_dtype) && vec_rows(x, ldx, x_dtype) &&
          vec_rows(dx, lddx, x_dtype) && aligned(weight, 16);
  a.w = weight;
  a.w_bf16 = w_dtype == HIF4_BF16;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.parts = sums ? (float*)workspace : nullptr;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_layer_norm_backward(a, x_dtype == HIF4_BF16, dweight, dbias, stream));
}

}  // extern "C"
