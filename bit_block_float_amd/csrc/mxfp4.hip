// mxfp4.hip -- quantize to the 4-bit microscaled format (E2M1 elements, a
// power-of-two scale per 32) and back. HBM-streaming kernels for gfx950.
//
// The scale is the smallest power of two s with amax <= 6 s, held as an E8M0 byte,
// so x / s is exact and encoding rounds once; the matrix cores apply the scale
// themselves (v_mfma_scale_f32_*).
//
// Bound: HBM. Along the rows 2 (bf16) or 4 (fp32) bytes are read and 1/2 + 1/32
// written an element; the tile kernel reads a 128 x 128 tile once for codes along the
// columns, or along both (what the two products of a linear layer's backward read).
#include "mxfp4_dev.h"

namespace hif4 {

// Over lanes l, l ^ 16, l ^ 32 and l ^ 48, by permlane swaps (no LDS permutes).
__device__ __forceinline__ uint32_t max_rows16(uint32_t v) {
  auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(p[0], p[1]);
  p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(p[0], p[1]);
}

// Along k. One lane owns 16 consecutive elements, two lanes a block; 8 lanes form a
// word of four scales, which the products read as one. One item a thread, all of a
// launch's reads independent: 57600 x 5120 bf16 126 to 150 us from box to box (5.0 to
// 5.9 TB/s; a copy 5.0 to 5.2).
template <typename T, int kRows>
__global__ __launch_bounds__(256) void quantize_mxfp4_rows_kernel(
    const T* __restrict__ x, int64_t ld, int k, uint32_t items_per_row, FastDiv item_div,
    uint32_t total_items, uint2* __restrict__ codes, uint32_t* __restrict__ scales) {
  const uint32_t it = blockIdx.x * 256u + threadIdx.x;
  if (it >= total_items) return;  // whole scale words: items_per_row is a multiple of 8
  const uint32_t row = fdiv(it, item_div);
  const uint32_t j = it - row * items_per_row;
  const T* src = x + (int64_t)row * ld;
  Run8<T> r0, r1;
  r0.template load<kRows>(src, (int)j * 16, k);
  r1.template load<kRows>(src, (int)j * 16 + 8, k);
  uint32_t m = max(r0.abs_max(), r1.abs_max());
  m = max(m, dpp<kDppQuadXor1>(m));
  const uint32_t e = mx4_scale_of(m);
  codes[it] = make_uint2(mx4_encode(r0, e), mx4_encode(r1, e));
  const uint32_t word = or8_u32(e << (8 * ((j >> 1) & 3u)));
  if ((j & 7u) == 0u) scales[it >> 3] = word;
}

// One tile of 128 rows x 128 columns a workgroup; the rows are those of a unit (128
// rows, or what is left of their group). Thread t holds rows 8 (t / 16) .. + 7 of
// columns 8 (t % 16) .. + 7, so a wave holds a block's 32 rows of 128 columns. The
// transposed codes go through LDS to leave as runs of 64 bytes, half a line, which the
// L2 joins for most (16384 x 2048: 46 MB reach memory of 38). Measured, both ways: 8192 x
// 5120 bf16 31 to 33 us (4.0 TB/s), 16384 x 2048 in 16 groups 26 to 28; along the rows
// only, 4099 x 1300 fp32 in 7 groups 9.2, 418 workgroups of one latency.
//  kAlong: codes [rows][ceil(k/128)*64], scales [rows][ceil(k/128)*4].
//  kCols: codes_t [k][units*64], scales_t [k][units*4] of batch number blockIdx.y.
//  unit0: the launch's first unit; units behind the last group are written as zeros.
template <typename T, bool kAlong, bool kCols, int kRows>
__global__ __launch_bounds__(256) void quantize_mxfp4_tile_kernel(
    const T* __restrict__ x, int64_t ld, int64_t rows, int k, int64_t unit0, int64_t units,
    uint32_t tiles_k, Groups groups, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
    uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t) {
  constexpr int kPitch = 17;  // words a column: 8 columns apart start 8 banks apart
  __shared__ uint32_t tile[kCols ? 128 * kPitch : 1];
  __shared__ uint8_t part[kCols ? 128 * 4 : 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid & 15, rg = tid >> 4;
  const uint32_t in = blockIdx.x / tiles_k;
  const int64_t unit = unit0 + in, b = blockIdx.y;
  const int tk = (int)(blockIdx.x - in * tiles_k);
  const int col0 = tk * 128 + cg * 8;
  int64_t begin = unit * 128, end = min(begin + 128, rows);
  if (groups.offsets) {
    int e;
    uint32_t before;
    if (group_unit(groups, 7, (uint32_t)unit, e, before)) {
      group_range(groups, e, begin, end);
      begin += (unit - before) * 128;
      end = min(begin + 128, end);
    } else {
      begin = end = 0;
    }
  }
  Run8<T> v[8];
  const T* src = x + b * rows * ld;
  if (begin + 128 == end && tk * 128 + 128 <= k) {  // a whole tile
    src += (begin + rg * 8) * ld + col0;
#pragma unroll
    for (int r = 0; r < 8; ++r) load_whole<kRows>(v[r], src + r * ld);
  } else if (begin < end) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
      v[r].template load<kRows>(src + min(begin + rg * 8 + r, end - 1) * ld, col0, k);
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r].keep_if(begin + rg * 8 + r < end);
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = Run8<T>{};
  }
  if constexpr (kAlong) {
    const int64_t at = (b * rows + begin + rg * 8) * tiles_k + tk;
    uint32_t* const c = reinterpret_cast<uint32_t*>(codes + at * 64) + cg;
    uint32_t* const sc = reinterpret_cast<uint32_t*>(scales) + at;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t m = v[r].abs_max();
      m = max(m, dpp<kDppQuadXor1>(m));
      m = max(m, dpp<kDppQuadXor2>(m));
      const uint32_t e = mx4_scale_of(m);
      uint32_t word = or8_u32(e << (8 * (cg >> 2)));
      word |= dpp<0x140>(word);  // row_mirror: over 16 lanes
      const uint32_t code = mx4_encode(v[r], e);
      if (begin + rg * 8 + r < end) {
        c[(int64_t)r * tiles_k * 16] = code;
        if (cg == 0) sc[(int64_t)r * tiles_k] = word;
      }
    }
  }
  if constexpr (kCols) {
    uint32_t cm[8];
    column_max(v, cm);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = mx4_scale_of(max_rows16(cm[i]));
      tile[(cg * 8 + i) * kPitch + rg] = mx4_encode_column(v, i, e);
      if (lane < 16) part[(cg * 8 + i) * 4 + wave] = (uint8_t)e;
    }
    __syncthreads();
    const int64_t row_t = b * k + (int64_t)tk * 128;  // of the transpose
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int c = p * 64 + (tid >> 2), q = tid & 3;
      const uint32_t* s = tile + c * kPitch + q * 4;
      if (tk * 128 + c < k)
        *reinterpret_cast<uint4*>(codes_t + ((row_t + c) * units + unit) * 64 + q * 16) =
            make_uint4(s[0], s[1], s[2], s[3]);
    }
    if (tid < 128 && tk * 128 + tid < k) {
      const uint8_t* s = part + tid * 4;
      *reinterpret_cast<uint32_t*>(scales_t + ((row_t + tid) * units + unit) * 4) =
          s[0] | (uint32_t)s[1] << 8 | (uint32_t)s[2] << 16 | (uint32_t)s[3] << 24;
    }
  }
}

// Codes back to values: 8 elements a thread, exact in either type (a value beyond the
// type's range becomes infinite). Bound: HBM, 1/2 + 1/32 bytes in and 2 or 4 out:
// 57600 x 5120 to bf16 123 to 128 us (5.9 TB/s). A NaN scale is or-ed in: a select with
// branches took 5% more.
template <bool kBf16>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint32_t runs_per_row,
    FastDiv run_div, uint32_t total, uint32_t words_per_row, int k,
    void* __restrict__ out) {
  const uint32_t it = blockIdx.x * 256u + threadIdx.x;
  if (it >= total) return;
  const uint32_t row = fdiv(it, run_div);
  const uint32_t j = it - row * runs_per_row;
  const int64_t at = (int64_t)row * words_per_row + j;
  const uint32_t w = codes[at], e = scales[at >> 2];
  const float s = mx4_scale(e);
  const uint32_t nan = e == 255u ? 0x7FC07FC0u : 0u;  // or-ed to the values, in either type
  const int64_t off = (int64_t)row * k + j * 8;
  const int valid = k - (int)j * 8;
  if constexpr (kBf16) {
    uint32_t h[4] = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] |= nan;
    uint16_t* o = reinterpret_cast<uint16_t*>(out) + off;
    if (valid >= 8) {  // (whole 16-byte stores at any alignment of the row)
      __builtin_memcpy(o, h, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) o[i] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float v[8];
    const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
    const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    v[0] = p0[0], v[1] = p0[1], v[2] = p1[0], v[3] = p1[1];
    v[4] = p2[0], v[5] = p2[1], v[6] = p3[0], v[7] = p3[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) | nan);
    float* o = reinterpret_cast<float*>(out) + off;
    if (valid >= 8) {
      __builtin_memcpy(o, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) o[i] = v[i];
    }
  }
}

template <typename T, int kRows>
static hipError_t launch_mx4(const T* x, int64_t batch, int64_t rows, int64_t k, int64_t ld,
                             const Groups& groups, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                             uint8_t* scales_t, hipStream_t stream) {
  const int64_t tiles_k = (k + 127) / 128;
  if (!codes_t) {  // matrices of a batch follow one another: more rows
    const uint32_t ipr = (uint32_t)(tiles_k * 8);
    const FastDiv fd = make_fastdiv(ipr);
    const int64_t all = batch * rows, max_rows = ((int64_t)1 << 30) / ipr;  // item indices stay below 2^31
    for (int64_t r0 = 0; r0 < all; r0 += max_rows) {
      const int64_t nr = all - r0 < max_rows ? all - r0 : max_rows;
      const uint32_t total = (uint32_t)(nr * ipr);
      hipLaunchKernelGGL((quantize_mxfp4_rows_kernel<T, kRows>), dim3((total + 255) / 256), dim3(256),
                         0, stream, x + r0 * ld, ld, (int)k, ipr, fd, total,
                         reinterpret_cast<uint2*>(codes + r0 * tiles_k * 64),
                         reinterpret_cast<uint32_t*>(scales + r0 * tiles_k * 4));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int64_t units = groups.offsets ? most_units(rows, groups.count, 7) : (rows + 127) / 128;
  const int64_t max_batch = batch < 32768 ? batch : 32768;  // grid.y
  const int64_t max_units = ((int64_t)1 << 23) / tiles_k;  // a grid has fewer than 2^32 threads a side
  for (int64_t b0 = 0; b0 < batch; b0 += max_batch) {
    const int64_t nb = batch - b0 < max_batch ? batch - b0 : max_batch;
    const T* xb = x + b0 * rows * ld;
    uint8_t* const cb = codes ? codes + b0 * rows * tiles_k * 64 : nullptr;
    uint8_t* const sb = scales ? scales + b0 * rows * tiles_k * 4 : nullptr;
    uint8_t* const ct = codes_t + b0 * k * units * 64;
    uint8_t* const st = scales_t + b0 * k * units * 4;
    for (int64_t u0 = 0; u0 < units; u0 += max_units) {
      const int64_t nu = units - u0 < max_units ? units - u0 : max_units;
      const dim3 grid((unsigned)(nu * tiles_k), (unsigned)nb), block(256);
      if (codes)
        hipLaunchKernelGGL((quantize_mxfp4_tile_kernel<T, true, true, kRows>), grid, block, 0, stream,
                           xb, ld, rows, (int)k, u0, units, (uint32_t)tiles_k, groups, cb, sb, ct, st);
      else
        hipLaunchKernelGGL((quantize_mxfp4_tile_kernel<T, false, true, kRows>), grid, block, 0, stream,
                           xb, ld, rows, (int)k, u0, units, (uint32_t)tiles_k, groups, cb, sb, ct, st);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace hif4

using namespace hif4;

hipError_t hif4_launch_quantize_mxfp4(const void* x, bool bf16, int64_t batch, int64_t rows, int64_t k,
                                      int64_t ld, const Groups& groups, uint8_t* codes,
                                      uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                                      hipStream_t stream) {
  const int64_t piece = bf16 ? 8 : 4;
  const bool vec = ((uintptr_t)x & 15) == 0 && ld % piece == 0 && k % piece == 0;
#define HIF4_QUANTIZE(T, mode) \
  launch_mx4<T, mode>((const T*)x, batch, rows, k, ld, groups, codes, scales, codes_t, scales_t, stream)
  if (vec) return bf16 ? HIF4_QUANTIZE(uint16_t, kAligned) : HIF4_QUANTIZE(float, kAligned);
  if (k >= 8) return bf16 ? HIF4_QUANTIZE(uint16_t, kAny) : HIF4_QUANTIZE(float, kAny);
  return bf16 ? HIF4_QUANTIZE(uint16_t, kTiny) : HIF4_QUANTIZE(float, kTiny);
#undef HIF4_QUANTIZE
}

hipError_t hif4_launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                        int64_t k, void* out, bool out_bf16, hipStream_t stream) {
  const int64_t wpr = (k + 127) / 128 * 16;  // words of 8 codes a row
  const uint32_t rpr = (uint32_t)((k + 7) / 8);
  const FastDiv fd = make_fastdiv(rpr);
  const int64_t max_rows = ((int64_t)1 << 30) / rpr;
  for (int64_t r0 = 0; r0 < rows; r0 += max_rows) {
    const int64_t nr = rows - r0 < max_rows ? rows - r0 : max_rows;
    const uint32_t total = (uint32_t)(nr * rpr);
    const dim3 grid((total + 255) / 256), block(256);
    void* o = (char*)out + r0 * k * (out_bf16 ? 2 : 4);
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes) + r0 * wpr;
    const uint8_t* s = scales + r0 * wpr / 4;
    if (out_bf16)
      hipLaunchKernelGGL(dequantize_mxfp4_kernel<true>, grid, block, 0, stream, c, s, rpr, fd, total,
                         (uint32_t)wpr, (int)k, o);
    else
      hipLaunchKernelGGL(dequantize_mxfp4_kernel<false>, grid, block, 0, stream, c, s, rpr, fd, total,
                         (uint32_t)wpr, (int)k, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
