// api_fp8.hip -- the C ABI of the 8-bit (E4M3, block-scaled) linear layer,
// declared and documented in include/hif4.h. Every argument check runs before
// any HIP call.
#include <stdint.h>

#include "api_util.h"
#include "fp8_dev.h"

namespace {

int64_t up128(int64_t v) { return (v + 127) / 128 * 128; }

constexpr int64_t kMaxK = int64_t(1) << 22;  // rows of one tile stay within 32-bit offsets

hif4_status check_quantize(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ld,
                           int64_t block_rows) {
  if (rows < 0 || k < 0 || ld < k || rows >= (int64_t(1) << 31) || k > kMaxK) return HIF4_ERR_SHAPE;
  if (x_dtype != HIF4_F32 && x_dtype != HIF4_BF16) return HIF4_ERR_DTYPE;
  if (block_rows != 1 && block_rows != 128) return HIF4_ERR_ARG;
  if ((up128(rows) / 128) * (up128(k) / 128) >= (int64_t(1) << 31)) return HIF4_ERR_SHAPE;
  if (rows == 0 || k == 0) return HIF4_OK;
  if (!x) return HIF4_ERR_NULL;
  if (!aligned(x, x_dtype == HIF4_BF16 ? 2 : 4)) return HIF4_ERR_ALIGN;
  return HIF4_OK;
}

}  // namespace

extern "C" {

hif4_status hif4_quantize_fp8(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ld,
                              int64_t block_rows, int transposed, uint8_t* codes, uint8_t* scales,
                              int64_t lds, hipStream_t stream) {
  hif4_status st = check_quantize(x, x_dtype, rows, k, ld, block_rows);
  if (st != HIF4_OK) return st;
  if (transposed != 0 && transposed != 1) return HIF4_ERR_ARG;
  if (rows == 0 || k == 0) return HIF4_OK;
  if (!codes || !scales) return HIF4_ERR_NULL;
  if (lds < (transposed ? up128(rows) : up128(k)) / 128) return HIF4_ERR_SHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 4) || lds % 4 != 0) return HIF4_ERR_ALIGN;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_quantize_fp8(
      x, x_dtype == HIF4_BF16, rows, k, ld, (int)block_rows, transposed ? nullptr : codes,
      transposed ? nullptr : scales, lds, transposed ? codes : nullptr,
      transposed ? scales : nullptr, lds, stream));
}

hif4_status hif4_quantize_fp8_both(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ld,
                                   int64_t block_rows, uint8_t* codes, uint8_t* scales, int64_t lds,
                                   uint8_t* codes_t, uint8_t* scales_t, int64_t lds_t,
                                   hipStream_t stream) {
  hif4_status st = check_quantize(x, x_dtype, rows, k, ld, block_rows);
  if (st != HIF4_OK) return st;
  if (rows == 0 || k == 0) return HIF4_OK;
  if (!codes || !scales || !codes_t || !scales_t) return HIF4_ERR_NULL;
  if (lds < up128(k) / 128 || lds_t < up128(rows) / 128) return HIF4_ERR_SHAPE;
  if (!aligned(codes, 16) || !aligned(codes_t, 16) || !aligned(scales, 4) ||
      !aligned(scales_t, 4) || lds % 4 != 0 || lds_t % 4 != 0)
    return HIF4_ERR_ALIGN;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_quantize_fp8(x, x_dtype == HIF4_BF16, rows, k, ld, (int)block_rows,
                                           codes, scales, lds, codes_t, scales_t, lds_t, stream));
}

hif4_status hif4_dequantize_fp8(const uint8_t* codes, const void* scales, int scale_type,
                                int64_t block_rows, int64_t lds, int64_t rows, int64_t k, void* out,
                                int out_dtype, hipStream_t stream) {
  if (rows < 0 || k < 0 || rows >= (int64_t(1) << 31) || k > kMaxK) return HIF4_ERR_SHAPE;
  if (out_dtype != HIF4_F32 && out_dtype != HIF4_BF16) return HIF4_ERR_DTYPE;
  if (scale_type != HIF4_SCALE_E8M0 && scale_type != HIF4_SCALE_F32) return HIF4_ERR_DTYPE;
  if (block_rows != 1 && block_rows != 128) return HIF4_ERR_ARG;
  if (rows == 0 || k == 0) return HIF4_OK;
  if (!codes || !scales || !out) return HIF4_ERR_NULL;
  if (lds < up128(k) / 128) return HIF4_ERR_SHAPE;
  if (!aligned(codes, 16) || !aligned(out, out_dtype == HIF4_BF16 ? 2 : 4) ||
      !aligned(scales, scale_type == HIF4_SCALE_F32 ? 4 : 1))
    return HIF4_ERR_ALIGN;
  hif4_status st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_dequantize_fp8(codes, scales, scale_type == HIF4_SCALE_F32,
                                             (int)block_rows, lds, rows, k, out,
                                             out_dtype == HIF4_BF16, stream));
}

}  // extern "C"

namespace {

// The sizes that a product takes.
bool linear_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0 || k % 128 != 0 || m >= (int64_t(1) << 31) ||
      n >= (int64_t(1) << 31) || k > kMaxK)
    return false;
  // Grids have fewer than 2^32 threads: 256 a tile of 128 x 128 (smaller tiles are
  // for products of few tiles, larger ones have no more threads for their size).
  return (m + 127) / 128 * ((n + 127) / 128) < (int64_t(1) << 24);
}

// Argument checks of a product, and the product of checked arguments.
hif4_status check_linear(const uint8_t* x_codes, const uint8_t* x_scales, int64_t ldxs,
                         const uint8_t* w_codes, const void* w_scales, int64_t ldws,
                         int w_scale_type, int64_t w_block_rows, int64_t m, int64_t n, int64_t k,
                         const void* y, int y_dtype, const void* workspace,
                         size_t workspace_bytes) {
  if (!linear_sizes(m, n, k)) return HIF4_ERR_SHAPE;
  if (y_dtype != HIF4_F32 && y_dtype != HIF4_BF16) return HIF4_ERR_DTYPE;
  if (w_scale_type != HIF4_SCALE_E8M0 && w_scale_type != HIF4_SCALE_F32) return HIF4_ERR_DTYPE;
  if (w_block_rows != 1 && w_block_rows != 128) return HIF4_ERR_ARG;
  if (w_scale_type == HIF4_SCALE_F32 && w_block_rows != 128) return HIF4_ERR_ARG;
  if (m == 0 || n == 0) return HIF4_OK;
  if (!y) return HIF4_ERR_NULL;
  if (!aligned(y, 16)) return HIF4_ERR_ALIGN;
  if (k == 0) return HIF4_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales) return HIF4_ERR_NULL;
  if (ldxs < k / 128 || ldws < k / 128 || ldxs > kMaxK || ldws > kMaxK) return HIF4_ERR_SHAPE;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 4) ||
      !aligned(w_scales, 4) || ldxs % 4 != 0 ||
      (w_scale_type == HIF4_SCALE_E8M0 && ldws % 4 != 0))
    return HIF4_ERR_ALIGN;
  const size_t need = hif4_gemm_fp8_ws_bytes(m, n, k);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return HIF4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HIF4_ERR_ALIGN;
  }
  return HIF4_OK;
}

hif4_status run_linear(const uint8_t* x_codes, const uint8_t* x_scales, int64_t ldxs,
                       const uint8_t* w_codes, const void* w_scales, int64_t ldws, int w_scale_type,
                       int64_t w_block_rows, int64_t m, int64_t n, int64_t k, void* y, int y_dtype,
                       void* workspace, hipStream_t stream) {
  if (m == 0 || n == 0) return HIF4_OK;
  if (k == 0) {
    // Empty contraction: Y = 0.
    const size_t bytes = (size_t)m * (size_t)n * (y_dtype == HIF4_BF16 ? 2 : 4);
    return launched(hif4_launch_zero(y, bytes, stream));
  }
  return launched(hif4_launch_gemm_fp8(
      Fp8Product{x_codes, x_scales, ldxs, w_codes, w_scales, ldws, w_scale_type == HIF4_SCALE_F32,
                 (int)w_block_rows, m, n, k, y, y_dtype == HIF4_BF16},
      workspace, stream));
}

}  // namespace

extern "C" {

size_t hif4_linear_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return linear_sizes(m, n, k) ? hif4_gemm_fp8_ws_bytes(m, n, k) : 0;
}

hif4_status hif4_linear_fp8(const uint8_t* x_codes, const uint8_t* x_scales, int64_t ldxs,
                            const uint8_t* w_codes, const void* w_scales, int64_t ldws,
                            int w_scale_type, int64_t w_block_rows, int64_t m, int64_t n, int64_t k,
                            void* y, int y_dtype, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  hif4_status st = check_linear(x_codes, x_scales, ldxs, w_codes, w_scales, ldws, w_scale_type,
                                w_block_rows, m, n, k, y, y_dtype, workspace, workspace_bytes);
  if (st != HIF4_OK || m == 0 || n == 0) return st;
  st = check_device();
  if (st != HIF4_OK) return st;
  return run_linear(x_codes, x_scales, ldxs, w_codes, w_scales, ldws, w_scale_type, w_block_rows, m,
                    n, k, y, y_dtype, workspace, stream);
}

// Workspace of the backward, each part 256-byte aligned: dY's codes [m][np] and
// scales [m][lds], its transposed codes [n][mp] and scales [n][lds_t], and what
// the larger product needs.
namespace {
// The sizes that a backward takes: those of dY's quantization and of both products.
bool backward_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0 || m > kMaxK || n > kMaxK || k >= (int64_t(1) << 31)) return false;
  return linear_sizes(m, k, up128(n)) && linear_sizes(n, k, up128(m));
}

struct BackwardParts {
  int64_t np, mp, lds, lds_t;
  size_t scales, codes_t, scales_t, product, total;
};
BackwardParts backward_parts(int64_t m, int64_t n, int64_t k) {
  BackwardParts p;
  p.np = up128(n);
  p.mp = up128(m);
  p.lds = (p.np / 128 + 3) / 4 * 4;
  p.lds_t = (p.mp / 128 + 3) / 4 * 4;
  p.scales = align256((size_t)m * (size_t)p.np);
  p.codes_t = p.scales + align256((size_t)m * (size_t)p.lds);
  p.scales_t = p.codes_t + align256((size_t)n * (size_t)p.mp);
  p.product = p.scales_t + align256((size_t)n * (size_t)p.lds_t);
  const size_t a = hif4_gemm_fp8_ws_bytes(m, k, p.np);
  const size_t b = hif4_gemm_fp8_ws_bytes(n, k, p.mp);
  p.total = p.product + align256(a > b ? a : b);
  return p;
}
}  // namespace

size_t hif4_linear_fp8_backward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return backward_sizes(m, n, k) ? backward_parts(m, n, k).total : 0;
}

hif4_status hif4_linear_fp8_backward(const void* dy, int dy_dtype, int64_t lddy,
                                     const uint8_t* xt_codes, const uint8_t* xt_scales,
                                     int64_t ldxt, const uint8_t* wt_codes, const void* wt_scales,
                                     int64_t ldwt, int wt_scale_type, int64_t wt_block_rows,
                                     int64_t m, int64_t n, int64_t k, void* dx, int dx_dtype,
                                     void* dw, int dw_dtype, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  if (!backward_sizes(m, n, k)) return HIF4_ERR_SHAPE;
  hif4_status st = check_quantize(dy, dy_dtype, m, n, lddy, 1);
  if (st != HIF4_OK) return st;
  if ((dx_dtype != HIF4_F32 && dx_dtype != HIF4_BF16) ||
      (dw_dtype != HIF4_F32 && dw_dtype != HIF4_BF16))
    return HIF4_ERR_DTYPE;
  const BackwardParts p = backward_parts(m, n, k);
  char* const ws = (char*)workspace;
  if (m > 0 && n > 0 && k > 0 && (dx || dw)) {
    if (!workspace || workspace_bytes < p.total) return HIF4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HIF4_ERR_ALIGN;
  }
  const uint8_t* const codes = (const uint8_t*)ws;
  const uint8_t* const codes_t = (const uint8_t*)(ws + p.codes_t);
  // Both products' arguments are checked before anything is enqueued. (A missing
  // workspace is refused above wherever the products read it.)
  if (dx) {
    st = check_linear(codes, codes + p.scales, p.lds, wt_codes, wt_scales, ldwt, wt_scale_type,
                      wt_block_rows, m, k, p.np, dx, dx_dtype, ws + p.product, SIZE_MAX);
    if (st != HIF4_OK) return st;
  }
  if (dw) {
    st = check_linear(codes_t, (const uint8_t*)(ws + p.scales_t), p.lds_t, xt_codes, xt_scales, ldxt,
                      HIF4_SCALE_E8M0, 1, n, k, p.mp, dw, dw_dtype, ws + p.product, SIZE_MAX);
    if (st != HIF4_OK) return st;
  }
  if (!dx && !dw) return HIF4_OK;
  st = check_device();
  if (st != HIF4_OK) return st;
  if (m > 0 && n > 0 && k > 0) {
    st = launched(hif4_launch_quantize_fp8(
        dy, dy_dtype == HIF4_BF16, m, n, lddy, 1, dx ? (uint8_t*)ws : nullptr,
        dx ? (uint8_t*)ws + p.scales : nullptr, p.lds, dw ? (uint8_t*)ws + p.codes_t : nullptr,
        dw ? (uint8_t*)ws + p.scales_t : nullptr, p.lds_t, stream));
    if (st != HIF4_OK) return st;
  }
  if (dx && dw && m > 0 && n > 0 && k > 0) {
    // the longer tiles (fp32 dW's, where dX is bf16) first
    return launched(hif4_launch_gemm_fp8_two(
        Fp8Product{codes_t, (const uint8_t*)(ws + p.scales_t), p.lds_t, xt_codes, xt_scales, ldxt,
                   false, 1, n, k, p.mp, dw, dw_dtype == HIF4_BF16},
        Fp8Product{codes, codes + p.scales, p.lds, wt_codes, wt_scales, ldwt,
                   wt_scale_type == HIF4_SCALE_F32, (int)wt_block_rows, m, k, p.np, dx,
                   dx_dtype == HIF4_BF16},
        ws + p.product, stream));
  }
  if (dx) {
    st = run_linear(codes, codes + p.scales, p.lds, wt_codes, wt_scales, ldwt, wt_scale_type,
                    wt_block_rows, m, k, p.np, dx, dx_dtype, ws + p.product, stream);
    if (st != HIF4_OK) return st;
  }
  if (dw)
    st = run_linear(codes_t, (const uint8_t*)(ws + p.scales_t), p.lds_t, xt_codes, xt_scales, ldxt,
                    HIF4_SCALE_E8M0, 1, n, k, p.mp, dw, dw_dtype, ws + p.product, stream);
  return st;
}

}  // extern "C"
