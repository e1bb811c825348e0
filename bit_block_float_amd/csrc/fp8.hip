// fp8.hip -- quantize to E4M3 with one power-of-two scale per block of 128,
// and back. HBM-streaming kernels for gfx950.
//
// A block is 1 x 128 along the contraction (activations, gradients) or
// 128 x 128 (weights, whose transpose then has the same codes and scales). The
// scale is the smallest power of two s with amax <= 448 s, held as an E8M0
// byte: x / s is exact in fp32, so encoding rounds once, and the matrix cores
// apply the scale themselves (v_mfma_scale_f32_*).
//
// Bound: HBM. 1 x 128 along the rows reads 2 (bf16) or 4 (fp32) bytes and
// writes 1 + 1/128 per element; the tile kernel reads a 128 x 128 tile once
// for any of its outputs (codes along the rows, codes along the columns, or
// both, which is what the two products of a linear layer's backward read).
// Measured, bf16: rows 57600 x 5120 150 us (5.9 TB/s; a copy of as many bytes
// runs at 5.0); 13824 x 5120 in tiles, codes of the transpose, 39 us (5.4 TB/s);
// 8192 x 5120 both ways 36 us (4.7 TB/s).
#include "fp8_dev.h"

namespace hif4 {

__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {  // over 16 aligned lanes
  v = max8_u32(v);
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
}

// 1 x 128 blocks along k. One lane owns 16 consecutive elements, 8 aligned
// lanes a block; the block maximum is formed with DPP moves. One item a thread
// and no loop, as in quantize_kernel: workgroups retire and are replaced on
// whichever CUs run ahead.
template <typename T, int kRows>
__global__ __launch_bounds__(256) void quantize_fp8_rows_kernel(
    const T* __restrict__ x, int64_t ld, int k, uint32_t items_per_row, FastDiv item_div,
    uint32_t total_items, uint4* __restrict__ codes, uint8_t* __restrict__ scales,
    int64_t lds) {
  const uint32_t it = blockIdx.x * 256u + threadIdx.x;
  if (it >= total_items) return;  // whole blocks: items_per_row is a multiple of 8
  const uint32_t row = fdiv(it, item_div);
  const uint32_t j = it - row * items_per_row;
  const T* src = x + (int64_t)row * ld;
  Run8<T> r0, r1;
  r0.template load<kRows>(src, (int)j * 16, k);
  r1.template load<kRows>(src, (int)j * 16 + 8, k);
  const uint32_t e = e8m0_of(max8_u32(max(r0.abs_max(), r1.abs_max())));
  const uint2 c0 = r0.encode(e), c1 = r1.encode(e);
  const uint4 w = make_uint4(c0.x, c0.y, c1.x, c1.y);
  codes[it] = w;
  if ((j & 7u) == 0u) scales[(int64_t)row * lds + (j >> 3)] = (uint8_t)e;
}

// One 128 x 128 tile a workgroup. Thread t holds rows 8 (t / 16) .. + 7 of
// columns 8 (t % 16) .. + 7: a row's 128 columns are 16 consecutive lanes, and
// the 8 rows of a column are 8 consecutive bytes of the transposed codes,
// which go through LDS to leave as whole 128-byte lines.
//  kTile: one scale for the tile; else one per row (kAlong) or column (kCols).
//  kAlong: codes [rows][ceil(k/128)*128]; kCols: codes_t [k][ceil(rows/128)*128].
//  row_tile0: the launch's first row of tiles.
template <typename T, bool kTile, bool kAlong, bool kCols, int kRows>
__global__ __launch_bounds__(256) void quantize_fp8_tile_kernel(
    const T* __restrict__ x, int64_t ld, int64_t rows, int k, int64_t row_tile0, uint32_t tiles_k,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t lds,
    uint8_t* __restrict__ codes_t, uint8_t* __restrict__ scales_t, int64_t lds_t) {
  constexpr int kPitch = 128 + 16;  // 16-byte reads stay aligned, columns spread over banks
  __shared__ __attribute__((aligned(16))) uint8_t tile[kCols ? 128 * kPitch : 16];
  __shared__ uint32_t part[4][kTile ? 1 : 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid & 15, rg = tid >> 4;
  const uint32_t in = blockIdx.x / tiles_k;
  const int64_t tr = row_tile0 + in;
  const int tk = (int)(blockIdx.x - in * tiles_k);
  const int64_t row0 = tr * 128 + rg * 8;
  const int col0 = tk * 128 + cg * 8;
  Run8<T> v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r)
    v[r].template load<kRows>(x + min(row0 + r, rows - 1) * ld, col0, k);
#pragma unroll
  for (int r = 0; r < 8; ++r) v[r].keep_if(row0 + r < rows);
  uint32_t e_tile = 0;
  uint32_t e_col[8];
  if constexpr (kTile) {
    uint32_t am = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) am = max(am, v[r].abs_max());
    am = max16_u32(am);
    am = max(am, (uint32_t)__shfl_xor((int)am, 16, 64));
    am = max(am, (uint32_t)__shfl_xor((int)am, 32, 64));
    if (lane == 0) part[wave][0] = am;
    __syncthreads();
    e_tile = e8m0_of(max(max(part[0][0], part[1][0]), max(part[2][0], part[3][0])));
  } else if constexpr (kCols) {
    uint32_t cm[8];
    column_max(v, cm);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t am = cm[i];
      am = max(am, (uint32_t)__shfl_xor((int)am, 16, 64));
      am = max(am, (uint32_t)__shfl_xor((int)am, 32, 64));
      if (lane < 16) part[wave][cg * 8 + i] = am;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = cg * 8 + i;
      e_col[i] = e8m0_of(max(max(part[0][c], part[1][c]), max(part[2][c], part[3][c])));
    }
  }
  if constexpr (kAlong) {
    const int64_t kp = (int64_t)tiles_k * 128;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t e = e_tile;
      if constexpr (!kTile) e = e8m0_of(max16_u32(v[r].abs_max()));
      const uint2 w = v[r].encode(e);
      if (row0 + r < rows) {
        *reinterpret_cast<uint2*>(codes + (row0 + r) * kp + col0) = w;
        if (!kTile && cg == 0) scales[(row0 + r) * lds + tk] = (uint8_t)e;
      }
    }
    if (kTile && tid == 0) scales[tr * lds + tk] = (uint8_t)e_tile;
  }
  if constexpr (kCols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = kTile ? e_tile : e_col[i];
      const uint2 w = encode_column(v, i, e);
      *reinterpret_cast<uint2*>(tile + (cg * 8 + i) * kPitch + rg * 8) = w;
      if (!kTile && rg == 0 && col0 + i < k)
        scales_t[(int64_t)(col0 + i) * lds_t + tr] = (uint8_t)e;
    }
    if (kTile && tid == 0) scales_t[(int64_t)tk * lds_t + tr] = (uint8_t)e_tile;
    __syncthreads();
    const int64_t rp = (rows + 127) / 128 * 128;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int c = p * 32 + (tid >> 3), ch = tid & 7;
      const uint4 w = *reinterpret_cast<const uint4*>(tile + c * kPitch + ch * 16);
      if (tk * 128 + c < k)
        *reinterpret_cast<uint4*>(codes_t + (int64_t)(tk * 128 + c) * rp + tr * 128 + ch * 16) = w;
    }
  }
}

// Products c[i] s of code values and a float32 scale, to be rounded to bf16, made
// to round as the exact ones do. c s has up to 28 significant bits: rounded to fp32
// it may land on the middle between two bf16 values (16 low bits 0x8000) without
// being there, and only then a second rounding goes wrong. Such a product is moved
// one step to its own side of the middle; the double product is exact. (One branch
// for all 8: 57600 x 5120 take 160 us, with a branch each 172, unchecked 151.)
__device__ __forceinline__ void mul_for_bf16(float (&c)[8], float s) {
  float p[8];
  bool middle = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = c[i] * s;
    middle |= (__float_as_uint(p[i]) & 0xFFFFu) == 0x8000u;
  }
  if (middle) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double exact = fabs((double)c[i] * (double)s), held = fabs((double)p[i]);
      const uint32_t u = __float_as_uint(p[i]);
      if ((u & 0xFFFFu) == 0x8000u) p[i] = __uint_as_float(u + (exact > held) - (exact < held));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = p[i];
}

// Codes back to values: 8 elements a thread. The scale of element (r, j) is
// scales[r / block_rows][j / 128]. Bound: HBM, 1 byte in and 2 or 4 out: 57600 x 5120
// to bf16 145 us (6.1 TB/s; with float32 scales 160, see above), to fp32 391 us
// (3.8 TB/s).
template <bool kF32Scale, bool kBf16>
__global__ __launch_bounds__(256) void dequantize_fp8_kernel(
    const uint8_t* __restrict__ codes, const void* __restrict__ scales, int row_shift, int64_t row0,
    int64_t lds, uint32_t runs_per_row, FastDiv run_div, uint32_t total, int64_t kp, int k, bool vec,
    void* __restrict__ out) {
  const uint32_t it = blockIdx.x * 256u + threadIdx.x;
  if (it >= total) return;
  const uint32_t row = fdiv(it, run_div);
  const uint32_t j = it - row * runs_per_row;
  const uint2 w = *reinterpret_cast<const uint2*>(codes + (int64_t)row * kp + j * 8);
  const int64_t si = ((row0 + row) >> row_shift) * lds + (j >> 4);
  const float s = kF32Scale ? reinterpret_cast<const float*>(scales)[si]
                            : e8m0_f32(reinterpret_cast<const uint8_t*>(scales)[si]);
  float v[8];
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 0);
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 1);
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 2);
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 3);
  v[4] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 0);
  v[5] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 1);
  v[6] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 2);
  v[7] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 3);
  const int64_t off = (int64_t)row * k + j * 8;
  const int valid = k - (int)j * 8;
  if constexpr (kBf16) {
    if constexpr (kF32Scale) {
      mul_for_bf16(v, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= s;
    }
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = f32_to_bf16(v[i]);
    uint16_t* o = reinterpret_cast<uint16_t*>(out) + off;
    if (vec && valid >= 8) {
      *reinterpret_cast<uint4*>(o) = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16),
                                                h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) o[i] = (uint16_t)h[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    float* o = reinterpret_cast<float*>(out) + off;
    if (vec && valid >= 8) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) o[i] = v[i];
    }
  }
}

template <typename T, int kRows>
static hipError_t launch_quantize(const T* x, int64_t rows, int64_t k, int64_t ld, int block_rows,
                                  uint8_t* codes, uint8_t* scales, int64_t lds, uint8_t* codes_t,
                                  uint8_t* scales_t, int64_t lds_t, hipStream_t stream) {
  const int64_t tiles_k = (k + 127) / 128, kp = tiles_k * 128;
  if (block_rows == 1 && !codes_t) {
    const uint32_t ipr = (uint32_t)(kp / 16);
    const FastDiv fd = make_fastdiv(ipr);
    const int64_t max_rows = ((int64_t)1 << 30) / ipr;  // item indices stay below 2^31
    for (int64_t r0 = 0; r0 < rows; r0 += max_rows) {
      const int64_t nr = rows - r0 < max_rows ? rows - r0 : max_rows;
      const uint32_t total = (uint32_t)(nr * ipr);
      hipLaunchKernelGGL((quantize_fp8_rows_kernel<T, kRows>), dim3((total + 255) / 256), dim3(256),
                         0, stream, x + r0 * ld, ld, (int)k, ipr, fd, total,
                         reinterpret_cast<uint4*>(codes + r0 * kp), scales + r0 * lds, lds);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int64_t tiles_m = (rows + 127) / 128;
  const int64_t max_tiles_m = ((int64_t)1 << 23) / tiles_k;  // a grid has fewer than 2^32 threads
  const dim3 block(256);
  const uint32_t tk = (uint32_t)tiles_k;
  for (int64_t t0 = 0; t0 < tiles_m; t0 += max_tiles_m) {
    const int64_t nt = tiles_m - t0 < max_tiles_m ? tiles_m - t0 : max_tiles_m;
    const dim3 grid((unsigned)(nt * tiles_k));
#define HIF4_TILE(tile, r, c)                                                                     \
  hipLaunchKernelGGL((quantize_fp8_tile_kernel<T, tile, r, c, kRows>), grid, block, 0, stream, x,  \
                     ld, rows, (int)k, t0, tk, codes, scales, lds, codes_t, scales_t, lds_t)
    if (block_rows == 1) {
      if (codes) HIF4_TILE(false, true, true);
      else HIF4_TILE(false, false, true);
    } else if (codes_t) {
      if (codes) HIF4_TILE(true, true, true);
      else HIF4_TILE(true, false, true);
    } else {
      HIF4_TILE(true, true, false);
    }
#undef HIF4_TILE
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace hif4

using namespace hif4;

hipError_t hif4_launch_quantize_fp8(const void* x, bool bf16, int64_t rows, int64_t k, int64_t ld,
                                    int block_rows, uint8_t* codes, uint8_t* scales, int64_t lds,
                                    uint8_t* codes_t, uint8_t* scales_t, int64_t lds_t,
                                    hipStream_t stream) {
  const int64_t piece = bf16 ? 8 : 4;
  const bool vec = ((uintptr_t)x & 15) == 0 && ld % piece == 0 && k % piece == 0;
#define HIF4_QUANTIZE(T, mode)                                                                  \
  launch_quantize<T, mode>((const T*)x, rows, k, ld, block_rows, codes, scales, lds, codes_t,    \
                           scales_t, lds_t, stream)
  if (vec) return bf16 ? HIF4_QUANTIZE(uint16_t, kAligned) : HIF4_QUANTIZE(float, kAligned);
  if (k >= 8) return bf16 ? HIF4_QUANTIZE(uint16_t, kAny) : HIF4_QUANTIZE(float, kAny);
  return bf16 ? HIF4_QUANTIZE(uint16_t, kTiny) : HIF4_QUANTIZE(float, kTiny);
#undef HIF4_QUANTIZE
}

hipError_t hif4_launch_dequantize_fp8(const uint8_t* codes, const void* scales, bool scales_f32,
                                      int block_rows, int64_t lds, int64_t rows, int64_t k,
                                      void* out, bool out_bf16, hipStream_t stream) {
  const int64_t kp = (k + 127) / 128 * 128;
  const uint32_t rpr = (uint32_t)((k + 7) / 8);
  const FastDiv fd = make_fastdiv(rpr);
  const int shift = block_rows == 128 ? 7 : 0;
  const int64_t max_rows = ((int64_t)1 << 30) / rpr;
  const bool vec = ((uintptr_t)out & 15) == 0 && k % (out_bf16 ? 8 : 4) == 0;
  for (int64_t r0 = 0; r0 < rows; r0 += max_rows) {
    const int64_t nr = rows - r0 < max_rows ? rows - r0 : max_rows;
    const uint32_t total = (uint32_t)(nr * rpr);
    const dim3 grid((total + 255) / 256), block(256);
    void* o = (char*)out + r0 * k * (out_bf16 ? 2 : 4);
    const uint8_t* c = codes + r0 * kp;
#define HIF4_DEQ(f, b)                                                                         \
  hipLaunchKernelGGL((dequantize_fp8_kernel<f, b>), grid, block, 0, stream, c, scales, shift, \
                     r0, lds, rpr, fd, total, kp, (int)k, vec, o)
    if (scales_f32) {
      if (out_bf16) HIF4_DEQ(true, true);
      else HIF4_DEQ(true, false);
    } else {
      if (out_bf16) HIF4_DEQ(false, true);
      else HIF4_DEQ(false, false);
    }
#undef HIF4_DEQ
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
