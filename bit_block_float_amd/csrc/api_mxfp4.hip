// api_mxfp4.hip -- the C ABI of the 4-bit microscaled (MXFP4) linear layers, grouped
// by expert and not, declared and documented in include/hif4.h. Every argument check
// runs before any HIP call.
#include <stdint.h>

#include "api_util.h"
#include "mxfp4_dev.h"

namespace {

using hif4::Groups;
using hif4::most_units;

int64_t up128(int64_t v) { return (v + 127) / 128 * 128; }

constexpr int64_t kMaxK = int64_t(1) << 22;  // rows of one tile stay within 32-bit offsets
constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxGroups = int64_t(1) << 16;
constexpr int64_t kMaxTiles = int64_t(1) << 24;  // of 256 threads: a grid has fewer than 2^32

bool dtype_ok(int t) { return t == HIF4_F32 || t == HIF4_BF16; }
size_t elem(int t) { return t == HIF4_BF16 ? 2 : 4; }

// Columns of a transpose whose rows are quantized along the source's rows.
int64_t columns(int64_t rows, int64_t groups, bool grouped) {
  return grouped ? 128 * most_units(rows, groups, 7) : up128(rows);
}

hif4_status check_x(const void* x, int x_dtype, int64_t batch, int64_t rows, int64_t k, int64_t ld) {
  if (batch < 0 || rows < 0 || k < 0 || ld < k || rows >= kMaxRows || batch >= kMaxRows || k > kMaxK)
    return HIF4_ERR_SHAPE;
  if (batch * rows >= kMaxRows) return HIF4_ERR_SHAPE;
  if (!dtype_ok(x_dtype)) return HIF4_ERR_DTYPE;
  if (batch == 0 || rows == 0 || k == 0) return HIF4_OK;
  if (!x) return HIF4_ERR_NULL;
  return aligned(x, elem(x_dtype)) ? HIF4_OK : HIF4_ERR_ALIGN;
}

hif4_status check_groups(const int64_t* offsets, int64_t groups) {
  if (groups < 0 || groups > kMaxGroups) return HIF4_ERR_SHAPE;
  if (groups > 0 && !offsets) return HIF4_ERR_NULL;
  return aligned(offsets, 8) ? HIF4_OK : HIF4_ERR_ALIGN;
}

// Of quantization with groups: along the rows of one matrix.
hif4_status check_quantize_groups(const int64_t* offsets, int64_t groups, int64_t batch, int64_t rows) {
  if (!offsets && groups == 0) return HIF4_OK;
  const hif4_status st = check_groups(offsets, groups);
  if (st != HIF4_OK) return st;
  if (groups == 0 || batch != 1) return HIF4_ERR_ARG;
  return columns(rows, groups, true) < kMaxRows ? HIF4_OK : HIF4_ERR_SHAPE;
}

hif4_status check_codes(const void* codes, const void* scales) {
  if (!codes || !scales) return HIF4_ERR_NULL;
  return aligned(codes, 16) && aligned(scales, 4) ? HIF4_OK : HIF4_ERR_ALIGN;
}

// What a product takes: rows of both sides (tiles of its launch below the limit) and
// its depth.
bool sizes_ok(int64_t m, int64_t n, int64_t k) {
  return m >= 0 && n >= 0 && k >= 0 && k % 128 == 0 && m < kMaxRows && n < kMaxRows && k <= kMaxK &&
         up128(m) / 128 * (up128(n) / 128) < kMaxTiles;
}
bool grouped_sizes_ok(int64_t groups, int64_t m, int64_t n, int64_t k) {
  if (groups < 0 || groups > kMaxGroups || !sizes_ok(0, n, k) || m < 0 || m >= kMaxRows) return false;
  return groups * n < kMaxRows && most_units(m, groups, 6) * ((n + 63) / 64) < kMaxTiles;
}
bool depth_sizes_ok(int64_t groups, int64_t m, int64_t n, int64_t k) {
  if (!sizes_ok(m, n, k)) return false;
  return groups * (up128(m) / 128) * (up128(n) / 128) < kMaxTiles;
}

Mx4Product product(const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int64_t m,
                   int64_t n, int64_t k, void* y, int y_dtype, int mode, Groups groups) {
  return Mx4Product{x, xs, k / 2, w, ws, k / 2, m, n, k, y, y_dtype == HIF4_BF16, mode, groups};
}

hif4_status run(const Mx4Product& p, void* workspace, hipStream_t stream) {
  if (p.m == 0 || p.n == 0) return HIF4_OK;
  if (p.k == 0 && p.mode == kMx4Plain)  // an empty contraction: Y = 0
    return launched(hif4_launch_zero(p.y, (size_t)p.m * (size_t)p.n * (p.y_bf16 ? 2 : 4), stream));
  return launched(hif4_launch_gemm_mxfp4(p, workspace, stream));
}

}  // namespace

extern "C" {

int64_t hif4_mxfp4_columns(int64_t rows, int64_t groups) {
  if (rows < 0 || rows >= kMaxRows || groups < 0 || groups > kMaxGroups) return 0;
  return columns(rows, groups, groups > 0);
}

hif4_status hif4_quantize_mxfp4(const void* x, int x_dtype, int64_t batch, int64_t rows, int64_t k,
                                int64_t ld, int transposed, const int64_t* offsets, int64_t groups,
                                uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  hif4_status st = check_x(x, x_dtype, batch, rows, k, ld);
  if (st != HIF4_OK) return st;
  if (transposed != 0 && transposed != 1) return HIF4_ERR_ARG;
  if (!transposed && (offsets || groups)) return HIF4_ERR_ARG;
  st = check_quantize_groups(offsets, groups, batch, rows);
  if (st != HIF4_OK) return st;
  if (batch == 0 || k == 0 || (transposed ? columns(rows, groups, groups > 0) : rows) == 0) return HIF4_OK;
  st = check_codes(codes, scales);
  if (st != HIF4_OK) return st;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_quantize_mxfp4(
      x, x_dtype == HIF4_BF16, batch, rows, k, ld, Groups{offsets, (int)groups, rows},
      transposed ? nullptr : codes, transposed ? nullptr : scales, transposed ? codes : nullptr,
      transposed ? scales : nullptr, stream));
}

hif4_status hif4_quantize_mxfp4_both(const void* x, int x_dtype, int64_t batch, int64_t rows, int64_t k,
                                     int64_t ld, const int64_t* offsets, int64_t groups, uint8_t* codes,
                                     uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                                     hipStream_t stream) {
  hif4_status st = check_x(x, x_dtype, batch, rows, k, ld);
  if (st != HIF4_OK) return st;
  st = check_quantize_groups(offsets, groups, batch, rows);
  if (st != HIF4_OK) return st;
  if (batch == 0 || k == 0 || columns(rows, groups, groups > 0) == 0) return HIF4_OK;
  if (rows > 0) {
    st = check_codes(codes, scales);
    if (st != HIF4_OK) return st;
  }
  st = check_codes(codes_t, scales_t);
  if (st != HIF4_OK) return st;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_quantize_mxfp4(x, x_dtype == HIF4_BF16, batch, rows, k, ld,
                                             Groups{offsets, (int)groups, rows}, codes, scales, codes_t,
                                             scales_t, stream));
}

hif4_status hif4_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t k,
                                  void* out, int out_dtype, hipStream_t stream) {
  if (rows < 0 || k < 0 || rows >= kMaxRows || k >= kMaxRows) return HIF4_ERR_SHAPE;
  if (!dtype_ok(out_dtype)) return HIF4_ERR_DTYPE;
  if (rows == 0 || k == 0) return HIF4_OK;
  if (!out) return HIF4_ERR_NULL;
  hif4_status st = check_codes(codes, scales);
  if (st != HIF4_OK) return st;
  if (!aligned(out, elem(out_dtype))) return HIF4_ERR_ALIGN;
  st = check_device();
  if (st != HIF4_OK) return st;
  return launched(hif4_launch_dequantize_mxfp4(codes, scales, rows, k, out, out_dtype == HIF4_BF16, stream));
}

size_t hif4_linear_mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return sizes_ok(m, n, k) ? hif4_gemm_mxfp4_ws_bytes(m, n, k) : 0;
}

hif4_status hif4_linear_mxfp4(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                              const uint8_t* w_scales, int64_t m, int64_t n, int64_t k, void* y,
                              int y_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!sizes_ok(m, n, k)) return HIF4_ERR_SHAPE;
  if (!dtype_ok(y_dtype)) return HIF4_ERR_DTYPE;
  if (m == 0 || n == 0) return HIF4_OK;
  if (!y) return HIF4_ERR_NULL;
  if (!aligned(y, 16)) return HIF4_ERR_ALIGN;
  hif4_status st;
  if (k > 0) {
    st = check_codes(x_codes, x_scales);
    if (st == HIF4_OK) st = check_codes(w_codes, w_scales);
    if (st != HIF4_OK) return st;
    const size_t need = hif4_gemm_mxfp4_ws_bytes(m, n, k);
    if (need > 0) {
      if (!workspace || workspace_bytes < need) return HIF4_ERR_WORKSPACE;
      if (!aligned(workspace, 256)) return HIF4_ERR_ALIGN;
    }
  }
  st = check_device();
  if (st != HIF4_OK) return st;
  return run(product(x_codes, x_scales, w_codes, w_scales, m, n, k, y, y_dtype, kMx4Plain, Groups{}),
             workspace, stream);
}

hif4_status hif4_linear_mxfp4_grouped(const uint8_t* x_codes, const uint8_t* x_scales,
                                      const uint8_t* w_codes, const uint8_t* w_scales,
                                      const int64_t* offsets, int64_t groups, int64_t m, int64_t n,
                                      int64_t k, void* y, int y_dtype, hipStream_t stream) {
  if (!grouped_sizes_ok(groups, m, n, k)) return HIF4_ERR_SHAPE;
  if (!dtype_ok(y_dtype)) return HIF4_ERR_DTYPE;
  hif4_status st = check_groups(offsets, groups);
  if (st != HIF4_OK) return st;
  if (m == 0 || n == 0 || groups == 0) return HIF4_OK;
  if (!y) return HIF4_ERR_NULL;
  if (!aligned(y, 16)) return HIF4_ERR_ALIGN;
  if (k > 0) {
    st = check_codes(x_codes, x_scales);
    if (st == HIF4_OK) st = check_codes(w_codes, w_scales);
    if (st != HIF4_OK) return st;
  }
  st = check_device();
  if (st != HIF4_OK) return st;
  return run(product(x_codes, x_scales, w_codes, w_scales, m, n, k, y, y_dtype, kMx4Rows,
                     Groups{offsets, (int)groups, m}),
             nullptr, stream);
}

}  // extern "C"

// Workspace of a backward, each part 256-byte aligned: dY's codes [m][np/2] and scales
// [m][np/32], its transpose's codes [n][mp/2] and scales [n][mp/32], and what the
// larger product needs.
namespace {
struct BackwardParts {
  int64_t np, mp;
  size_t scales, codes_t, scales_t, product, total;
};
BackwardParts backward_parts(int64_t m, int64_t n, int64_t k, int64_t groups, bool grouped) {
  BackwardParts p;
  p.np = up128(n);
  p.mp = columns(m, groups, grouped);
  p.scales = align256((size_t)m * (size_t)p.np / 2);
  p.codes_t = p.scales + align256((size_t)m * (size_t)p.np / 32);
  p.scales_t = p.codes_t + align256((size_t)n * (size_t)p.mp / 2);
  p.product = p.scales_t + align256((size_t)n * (size_t)p.mp / 32);
  const size_t a = grouped ? 0 : hif4_gemm_mxfp4_ws_bytes(m, k, p.np);
  const size_t b = grouped ? 0 : hif4_gemm_mxfp4_ws_bytes(n, k, p.mp);
  p.total = p.product + align256(a > b ? a : b);
  return p;
}
bool backward_sizes(int64_t m, int64_t n, int64_t k, int64_t groups, bool grouped) {
  if (m < 0 || n < 0 || k < 0 || m >= kMaxRows || n > kMaxK || k >= kMaxRows) return false;
  if (!grouped) return m <= kMaxK && sizes_ok(m, k, up128(n)) && sizes_ok(n, k, up128(m));
  if (groups < 0 || groups > kMaxGroups) return false;
  return grouped_sizes_ok(groups, m, k, up128(n)) && depth_sizes_ok(groups, n, k, columns(m, groups, true));
}

// Both gradients; `groups.offsets` NULL: one weight.
hif4_status backward(const void* dy, int dy_dtype, int64_t lddy, const uint8_t* xt_codes,
                     const uint8_t* xt_scales, const uint8_t* wt_codes, const uint8_t* wt_scales,
                     bool grouped, Groups groups, int64_t m, int64_t n, int64_t k, void* dx, int dx_dtype,
                     void* dw, int dw_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!backward_sizes(m, n, k, groups.count, grouped)) return HIF4_ERR_SHAPE;
  hif4_status st = check_x(dy, dy_dtype, 1, m, n, lddy);
  if (st != HIF4_OK) return st;
  if (!dtype_ok(dx_dtype) || !dtype_ok(dw_dtype)) return HIF4_ERR_DTYPE;
  if (grouped) {
    st = check_groups(groups.offsets, groups.count);
    if (st != HIF4_OK) return st;
  }
  const BackwardParts p = backward_parts(m, n, k, groups.count, grouped);
  if (k == 0 || (grouped && groups.count == 0)) return HIF4_OK;
  const bool want_dx = dx && m > 0, want_dw = dw && n > 0;
  if (!want_dx && !want_dw) return HIF4_OK;
  if ((want_dx && !aligned(dx, 16)) || (want_dw && !aligned(dw, 16))) return HIF4_ERR_ALIGN;
  const bool read = m > 0 && n > 0;  // dY has elements
  if (read) {
    if (want_dx) st = check_codes(wt_codes, wt_scales);
    if (st == HIF4_OK && want_dw) st = check_codes(xt_codes, xt_scales);
    if (st != HIF4_OK) return st;
    if (!workspace || workspace_bytes < p.total) return HIF4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HIF4_ERR_ALIGN;
  }
  st = check_device();
  if (st != HIF4_OK) return st;
  uint8_t* const ws = (uint8_t*)workspace;
  uint8_t *const codes = ws, *const scales = ws + p.scales;
  uint8_t *const codes_t = ws + p.codes_t, *const scales_t = ws + p.scales_t;
  if (read) {
    st = launched(hif4_launch_quantize_mxfp4(dy, dy_dtype == HIF4_BF16, 1, m, n, lddy, groups,
                                             want_dx ? codes : nullptr, want_dx ? scales : nullptr,
                                             want_dw ? codes_t : nullptr, want_dw ? scales_t : nullptr,
                                             stream));
    if (st != HIF4_OK) return st;
  }
  const Mx4Product a = product(codes_t, scales_t, xt_codes, xt_scales, n, k, read ? p.mp : 0, dw, dw_dtype,
                               grouped ? kMx4Depth : kMx4Plain, groups);
  const Mx4Product b = product(codes, scales, wt_codes, wt_scales, m, k, read ? p.np : 0, dx, dx_dtype,
                               grouped ? kMx4Rows : kMx4Plain, groups);
  if (read && want_dx && want_dw)
    return launched(hif4_launch_gemm_mxfp4_two(a, b, ws + p.product, stream));
  if (want_dw) st = run(a, ws + p.product, stream);
  if (st == HIF4_OK && want_dx) st = run(b, ws + p.product, stream);
  return st;
}
}  // namespace

extern "C" {

size_t hif4_linear_mxfp4_backward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return backward_sizes(m, n, k, 0, false) ? backward_parts(m, n, k, 0, false).total : 0;
}

hif4_status hif4_linear_mxfp4_backward(const void* dy, int dy_dtype, int64_t lddy, const uint8_t* xt_codes,
                                       const uint8_t* xt_scales, const uint8_t* wt_codes,
                                       const uint8_t* wt_scales, int64_t m, int64_t n, int64_t k, void* dx,
                                       int dx_dtype, void* dw, int dw_dtype, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  return backward(dy, dy_dtype, lddy, xt_codes, xt_scales, wt_codes, wt_scales, false,
                  Groups{nullptr, 0, m}, m, n, k, dx, dx_dtype, dw, dw_dtype, workspace, workspace_bytes,
                  stream);
}

size_t hif4_linear_mxfp4_grouped_backward_workspace_bytes(int64_t groups, int64_t m, int64_t n, int64_t k) {
  return backward_sizes(m, n, k, groups, true) ? backward_parts(m, n, k, groups, true).total : 0;
}

hif4_status hif4_linear_mxfp4_grouped_backward(
    const void* dy, int dy_dtype, int64_t lddy, const uint8_t* xt_codes, const uint8_t* xt_scales,
    const uint8_t* wt_codes, const uint8_t* wt_scales, const int64_t* offsets, int64_t groups, int64_t m,
    int64_t n, int64_t k, void* dx, int dx_dtype, void* dw, int dw_dtype, void* workspace,
    size_t workspace_bytes, hipStream_t stream) {
  return backward(dy, dy_dtype, lddy, xt_codes, xt_scales, wt_codes, wt_scales, true,
                  Groups{offsets, (int)(groups < 0 || groups > kMaxGroups ? -1 : groups), m}, m, n, k, dx,
                  dx_dtype, dw, dw_dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
