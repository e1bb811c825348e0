// norm.hip -- layer norm over the rows of a matrix: forward, forward that ends
// in a quantizer (HiF4 or E4M3 blocks), and backward with the reduction of the
// weight's and bias' gradients. HBM-streaming kernels for gfx950.
//
// Forward: y = (x - mean) rstd w + b with rstd = (var + eps)^(-1/2). A row is
// held in registers from its one read (part of one of more than 16384 columns in
// scratch memory), so the variance is the mean of (x - mean)^2 over what was read,
// not a difference of two large sums.
// Backward, with xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum over rows of dy xhat,  db = sum over rows of dy.
// Statistics, sums and gradients are fp32; results are rounded once.
#include <algorithm>
#include <type_traits>

#include "fp8_dev.h"
#include "norm_dev.h"
#include "quant_dev.h"

namespace hif4 {

enum NormOut { kOutY = 0, kOutHif4 = 1, kOutFp8 = 2 };

// Sum over the lanes of a wave, the same bits in every lane: DPP moves inside
// each row of 16 lanes, then the rows by permlane swaps (which leave the two
// rows, or halves, of a pair in two registers): no LDS permutes.
__device__ __forceinline__ float row16_sum(float v) {
  auto f = [](uint32_t u) { return __uint_as_float(u); };
  v += f(dpp<kDppQuadXor1>(__float_as_uint(v)));
  v += f(dpp<kDppQuadXor2>(__float_as_uint(v)));
  v += f(dpp<kDppHalfMirror>(__float_as_uint(v)));
  return v + f(dpp<0x140>(__float_as_uint(v)));  // row_mirror
}
__device__ __forceinline__ float wave_sum(float v) {
  auto f = [](uint32_t u) { return __uint_as_float(u); };
  v = row16_sum(v);
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(p[0]) + f(p[1]);
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(p[0]) + f(p[1]);
}

// Sum over aligned groups of 8, 16, 32 or 64 lanes: the steps of wave_sum that stay
// inside one (so the same bits as over 64 lanes of which the others hold zero).
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  auto f = [](uint32_t u) { return __uint_as_float(u); };
  if constexpr (kLanes == 64) return wave_sum(v);
  if constexpr (kLanes == 8) {
    v += f(dpp<kDppQuadXor1>(__float_as_uint(v)));
    v += f(dpp<kDppQuadXor2>(__float_as_uint(v)));
    return v + f(dpp<kDppHalfMirror>(__float_as_uint(v)));
  }
  v = row16_sum(v);
  if constexpr (kLanes == 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(p[0]) + f(p[1]);
  }
  return v;
}

// Sum over a workgroup of 1024 threads. `slot` is LDS of 16 floats that no other
// sum in flight uses.
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  return row16_sum(slot[threadIdx.x & 15]);
}

// 8 weights or biases from column `col` (fp32 or bf16), 1 / 0 without one.
template <int kRows>
__device__ __forceinline__ void load_w8(const void* w, bool w_bf16, int col, int c, float fallback,
                                        float (&v)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fallback;
  } else if (w_bf16) {
    Run8<uint16_t> r;
    r.load<kRows>(reinterpret_cast<const uint16_t*>(w), col, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
  } else {
    Run8<float> r;
    r.load<kRows>(reinterpret_cast<const float*>(w), col, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
  }
}

// 8 values rounded to bf16.
__device__ __forceinline__ Run8<uint16_t> pack8(const float (&v)[8]) {
  Run8<uint16_t> r;
  r.w = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                   f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
  return r;
}

template <int kRows>
__device__ __forceinline__ void store_run8(uint16_t* p, int valid, const float (&v)[8]) {
  if constexpr (kRows == kAligned) {
    if (valid <= 0) return;
    *reinterpret_cast<uint4*>(p) = pack8(v).w;
  } else if (valid >= 8) {
    const uint4 w = pack8(v).w;
    __builtin_memcpy(p, &w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint16_t)f32_to_bf16(v[i]);
  }
}
template <int kRows>
__device__ __forceinline__ void store_run8(float* p, int valid, const float (&v)[8]) {
  if constexpr (kRows == kAligned) {
    if (valid <= 0) return;
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else if (valid >= 8) {
    __builtin_memcpy(p, v, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = v[i];
  }
}

// Item j (16 columns) of a row of results: as they are, to HiF4, or to E4M3.
template <typename T, int kOut, int kRows>
__device__ __forceinline__ void store_item(const NormArgs& a, float (&y)[2][8], int64_t row, int j,
                                           int c, uint32_t info) {
  const int col = j * 16;
  if constexpr (kOut == kOutY) {
    T* dst = reinterpret_cast<T*>(a.y) + row * a.ldy + col;
    store_run8<kRows>(dst, c - col, y[0]);
    store_run8<kRows>(dst + 8, c - col - 8, y[1]);
  } else if constexpr (kOut == kOutHif4) {
    uint4 v0 = pack8(y[0]).w, v1 = pack8(y[1]).w;
    if (a.mask) {
      keep_item_values(v0, v1, info, row, a.kept, a.n_mask);
      uint32_t z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t lo = (info >> (16 + 2 * i)) & 1u, hi = (info >> (17 + 2 * i)) & 1u;
        z[i] = ~((lo * 0x0000FFFFu) | (hi * 0xFFFF0000u));
      }
      v0 = make_uint4(v0.x & z[0], v0.y & z[1], v0.z & z[2], v0.w & z[3]);
      v1 = make_uint4(v1.x & z[4], v1.y & z[5], v1.z & z[6], v1.w & z[7]);
    }
    quantize_item(v0, v1, (uint32_t)j, (uint32_t)j,
                  reinterpret_cast<uint32_t*>(a.codes + row * (c / 2)), a.meta + row * (c / 64));
  } else {
    Run8<T> r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kRows != kAligned) {  // the padding of the last block (whole runs: below)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[h][i] = col + 8 * h + i < c ? y[h][i] : 0.0f;
      }
      if constexpr (sizeof(T) == 2) {
        r[h] = pack8(y[h]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[h].v[i] = y[h][i];
      }
      if constexpr (kRows == kAligned) r[h].keep_if(col + 8 * h < c);
    }
    const uint32_t e = e8m0_of(max8_u32(max(r[0].abs_max(), r[1].abs_max())));
    const uint2 c0 = r[0].encode(e), c1 = r[1].encode(e);
    *reinterpret_cast<uint4*>(a.codes + row * a.kp + col) = make_uint4(c0.x, c0.y, c1.x, c1.y);
    if ((j & 7) == 0) a.scales[row * a.lds + (j >> 3)] = (uint8_t)e;
  }
}

// 16 mask bytes as bits, and the inclusive sum over the lanes up to this one.
__device__ __forceinline__ uint32_t mask_bits(const uint8_t* p) {
  const uint4 mk = *reinterpret_cast<const uint4*>(p);
  return nonzero_bytes(mk.x) | (nonzero_bytes(mk.y) << 4) | (nonzero_bytes(mk.z) << 8) |
         (nonzero_bytes(mk.w) << 12);
}
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

// Sum of up to 16 values in the order of row16_sum over lanes 0, 1, ...
template <int N>
__device__ __forceinline__ float tree_sum(const float (&v)[N]) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = i < N ? v[i] : 0.0f;
  const float a = (t[0] + t[1]) + (t[2] + t[3]), b = (t[4] + t[5]) + (t[6] + t[7]);
  const float c = (t[8] + t[9]) + (t[10] + t[11]), d = (t[12] + t[13]) + (t[14] + t[15]);
  return (a + b) + (c + d);
}

// Forward that ends in a quantizer, many bf16 rows of 4097 to 6144 columns.
// A wave owns a row (its lanes items n * 64 + lane), so nothing in the row loop
// waits for another wave: the encoders need too many registers for the kernel
// below to hide its barriers and loads behind other rows. Weight and bias are in
// LDS as fp32 ([weight, bias][quarter of an item][item] 16-byte pieces, which
// consecutive lanes read without bank conflicts). The sums are taken in the order
// of the kernel below: a tree over the lanes for each run of 64 items, then a
// tree over the runs, so the results are the same bits. Bound: VALU issue (HiF4:
// 26 instructions an element, which at 4 cycles each fill 86% of the SIMDs' time; the
// plain norm of the kernel below has 13). Measured on 57600 x 5120: HiF4 215 to 245 us
// (3.3 TB/s), E4M3 176 us (5.0 TB/s, what a copy reaches).
template <int kItems, int kOut>
__global__ __launch_bounds__(512) void layer_norm_wave_kernel(NormArgs a) {
  extern __shared__ float4 affine[];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int c = a.c;
  const int items = kOut == kOutFp8 ? a.kp / 16 : (c + 15) / 16;
  for (int j = threadIdx.x; j < items; j += blockDim.x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float w[8], b[8];
      load_w8<kAligned>(a.w, a.w_bf16, j * 16 + 8 * h, c, 1.0f, w);
      load_w8<kAligned>(a.b, a.w_bf16, j * 16 + 8 * h, c, 0.0f, b);
      affine[(2 * h) * items + j] = make_float4(w[0], w[1], w[2], w[3]);
      affine[(2 * h + 1) * items + j] = make_float4(w[4], w[5], w[6], w[7]);
      affine[(4 + 2 * h) * items + j] = make_float4(b[0], b[1], b[2], b[3]);
      affine[(5 + 2 * h) * items + j] = make_float4(b[4], b[5], b[6], b[7]);
    }
  }
  uint32_t info[kItems] = {};
  if (kOut == kOutHif4 && a.mask) {
    uint32_t run = 0;
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int j = n * 64 + lane;
      const uint32_t m16 = j < items ? mask_bits(a.mask + (size_t)j * 16) : 0u;
      const uint32_t incl = wave_prefix(__popc(m16), lane);
      info[n] = (m16 << 16) | ((run + incl - __popc(m16)) & 0xFFFFu);
      run += (uint32_t)__shfl((int)incl, 63, 64);
    }
  }
  __syncthreads();

  const float fc = (float)c, inv_c = 1.0f / (float)c;
  const int64_t step = (int64_t)gridDim.x * waves;
  for (int64_t row = (int64_t)blockIdx.x * waves + (threadIdx.x >> 6); row < a.rows; row += step) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.x) + row * a.ld;
    Run8<uint16_t> r[kItems][2];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      r[n][0].template load<kAligned>(src, (n * 64 + lane) * 16, c);
      r[n][1].template load<kAligned>(src, (n * 64 + lane) * 16 + 8, c);
    }
    float part[kItems];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      part[n] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) part[n] += r[n][0].get(i) + r[n][1].get(i);
      part[n] = wave_sum(part[n]);
    }
    const float mean = tree_sum<kItems>(part) / fc;
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      float q[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        r[n][h].opaque();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = r[n][h].get(i) - mean;
          q[h] = fmaf(d, d, q[h]);
        }
      }
      const int col = (n * 64 + lane) * 16;
      part[n] = wave_sum((col < c ? q[0] : 0.0f) + (col + 8 < c ? q[1] : 0.0f));
    }
    const float rstd = 1.0f / sqrtf(tree_sum<kItems>(part) * inv_c + a.eps);
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int j = n * 64 + lane;
      if (j >= items) continue;  // whole quads / octets of lanes
      float y[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        r[n][h].opaque();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 w = affine[(2 * h + e) * items + j], b = affine[(4 + 2 * h + e) * items + j];
          const float* pw = &w.x;
          const float* pb = &b.x;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[h][4 * e + i] = fmaf((r[n][h].get(4 * e + i) - mean) * rstd, pw[i], pb[i]);
        }
      }
      store_item<uint16_t, kOut, kAligned>(a, y, row, j, c, info[n]);
    }
  }
}

// Forward of the widest rows (over 16384 columns): 1024 threads share a row, a
// lane owns items (16 consecutive elements) t, t + 1024, ..., the quantizers' own
// mapping, so 4 aligned lanes hold a HiF4 unit and 8 an E4M3 block when the row
// leaves through one of them. The value quantized is the one kOutY would store
// (rounded to bf16 for HiF4, to x's type for E4M3), so the codes are those of the
// two calls in turn.
//
// Bound: not by HBM. 64 columns a lane do not fit the 128 registers that 1024
// threads leave (380 to 932 bytes of scratch a lane), and weight and bias are read
// again for each row. Measured, 4096 rows of bf16: 20480 columns 480 us (0.7 TB/s),
// to HiF4 615, to E4M3 503; 65536 columns 778, 900 and 800 us; of 16384 columns, by
// the kernel below, 64 us.
template <typename T, int kItems, int kOut, int kRows>
__global__ __launch_bounds__(1024) void layer_norm_wide_kernel(NormArgs a) {
  constexpr int P = 1024;
  __shared__ float slots[2][P / 64];
  const int t = threadIdx.x;
  const int c = a.c;
  const int items = kOut == kOutFp8 ? a.kp / 16 : (c + 15) / 16;
  const T* x = reinterpret_cast<const T*>(a.x);

  // protected channels (HiF4): the item's mask bits and the rank of its first
  // masked channel, the same in every row
  uint32_t info[kItems];
  if constexpr (kOut == kOutHif4) {
    if (a.mask) {
      __shared__ uint32_t part[P / 64];
      uint32_t run = 0;
#pragma unroll
      for (int n = 0; n < kItems; ++n) {
        const int j = n * P + t;
        const uint32_t m16 = j < items ? mask_bits(a.mask + (size_t)j * 16) : 0u;
        const uint32_t cnt = __popc(m16), incl = wave_prefix(cnt, t & 63);
        if ((t & 63) == 63) part[t >> 6] = incl;
        __syncthreads();
        uint32_t base = run, total = 0;
        for (int w = 0; w < P / 64; ++w) {
          if (w < (t >> 6)) base += part[w];
          total += part[w];
        }
        __syncthreads();
        info[n] = (m16 << 16) | ((base + incl - cnt) & 0xFFFFu);
        run += total;
      }
    }
  }

  const float inv_c = 1.0f / (float)c;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* src = x + row * a.ld;
    Run8<T> r0[kItems], r1[kItems];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int col = (n * P + t) * 16;
      r0[n].template load<kRows>(src, col, c);
      r1[n].template load<kRows>(src, col + 8, c);
    }
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < kItems; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += r0[n].get(i) + r1[n].get(i);
    const float mean = row_sum(s, slots[0]) / (float)c;
    float q = 0.0f;
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int valid = c - (n * P + t) * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d0 = i < valid ? r0[n].get(i) - mean : 0.0f;
        const float d1 = i + 8 < valid ? r1[n].get(i) - mean : 0.0f;
        q = fmaf(d0, d0, q);
        q = fmaf(d1, d1, q);
      }
    }
    const float var = row_sum(q, slots[1]) * inv_c;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (kOut == kOutY && t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int j = n * P + t;
      if (j >= items) continue;  // whole quads / octets of lanes: items is a multiple of 4 / 8
      const int col = j * 16;
      float y[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float w[8], b[8];
        load_w8<kRows>(a.w, a.w_bf16, col + 8 * h, c, 1.0f, w);
        load_w8<kRows>(a.b, a.w_bf16, col + 8 * h, c, 0.0f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[h][i] = fmaf(((h ? r1[n] : r0[n]).get(i) - mean) * rstd, w[i], b[i]);
      }
      store_item<T, kOut, kRows>(a, y, row, j, c, info[n]);
    }
  }
}

// Forward of rows of up to 16384 columns. The block's T = blockDim.x threads (64
// times the waves that a row's items of 16 columns fill) own one item each, of R
// rows at a time: weight and bias stay in registers for all rows, where the
// kernel above reads them again for each (57600 x 5120: they are twice x's own
// bytes), and two barriers serve R rows. Everything else is as above. Bound: HBM, a
// row read and written once: 57600 x 5120 bf16 235 us (5.0 TB/s, what a copy reaches),
// 57600 x 13824 675 us (4.7 TB/s); 77 x 1003 fp32 4.8 us and 509 x 5120 to E4M3 5.5 us,
// which are a launch and the latency of one read.
//
// Rows of up to 512 columns leave most lanes of a wave without an item: groups of
// kLanes = 8, 16 or 32 lanes take a row each (kMulti: a row is the workgroup's, of
// several waves).
template <typename T, int R, int kOut, bool kMulti, int kRows, int kLanes>
__global__ __launch_bounds__(1024) void layer_norm_rows_kernel(NormArgs a) {
  __shared__ float slots[2][R][16];
  static_assert(!kMulti || kLanes == 64, "whole waves share a row");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = kMulti ? threadIdx.x : threadIdx.x & (kLanes - 1);  // the item
  const int waves = kMulti ? (int)(blockDim.x >> 6) : 1;
  const int groups = kMulti ? 1 : (int)blockDim.x / kLanes, group = kMulti ? 0 : (int)threadIdx.x / kLanes;
  const int c = a.c, col = t * 16;
  const int items = kOut == kOutFp8 ? a.kp / 16 : (c + 15) / 16;
  const bool live = t < items;

  uint32_t info = 0;
  if constexpr (kOut == kOutHif4) {
    if (a.mask) {
      __shared__ uint32_t part[16];
      const uint32_t m16 = live ? mask_bits(a.mask + col) : 0u;
      const uint32_t cnt = __popc(m16), incl = wave_prefix(cnt, lane);
      uint32_t base = incl - cnt;
      if constexpr (kLanes < 64) base -= (uint32_t)__shfl((int)base, 0, kLanes);
      if constexpr (kMulti) {
        if (lane == 63) part[wave] = incl;
        __syncthreads();
        for (int w = 0; w < wave; ++w) base += part[w];
      }
      info = (m16 << 16) | (base & 0xFFFFu);
    }
  }

  float w[2][8], b[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_w8<kRows>(a.w, a.w_bf16, col + 8 * h, c, 1.0f, w[h]);
    load_w8<kRows>(a.b, a.w_bf16, col + 8 * h, c, 0.0f, b[h]);
  }

  // sums over the row's threads, R at once; `slot` turns between the two
  auto row_sums = [&](float (&v)[R], int slot) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = lanes_sum<kLanes>(v[r]);
    if constexpr (kMulti) {
      if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) slots[slot][r][wave] = v[r];
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r)
        v[r] = row16_sum((lane & 15) < waves ? slots[slot][r][lane & 15] : 0.0f);
    }
  };

  const float fc = (float)c, inv_c = 1.0f / (float)c;
  const int64_t step = (int64_t)gridDim.x * groups * R;
  // rows past the end read the last one again and are not stored
  Run8<T> n0[R], n1[R];
  auto load_rows = [&](int64_t row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const T* src = reinterpret_cast<const T*>(a.x) + min(row0 + r * groups + group, a.rows - 1) * a.ld;
      n0[r].template load<kRows>(src, col, c);
      n1[r].template load<kRows>(src, col + 8, c);
    }
  };
  for (int64_t row0 = (int64_t)blockIdx.x * groups * R; row0 < a.rows; row0 += step) {
    load_rows(row0);
    float x[R][2][8], mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[r][0][i] = n0[r].get(i);
        x[r][1][i] = n1[r].get(i);
        mean[r] += x[r][0][i] + x[r][1][i];
      }
    }
    row_sums(mean, 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] /= fc;
      float q[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[r][h][i] -= mean[r];
          const float d = kRows == kAligned || col + 8 * h + i < c ? x[r][h][i] : 0.0f;
          q[h] = fmaf(d, d, q[h]);
        }
      // kAligned: a run is whole or empty
      rstd[r] = (kRows != kAligned || col < c ? q[0] : 0.0f) +
                (kRows != kAligned || col + 8 < c ? q[1] : 0.0f);
    }
    row_sums(rstd, 1);
#pragma unroll
    for (int r = 0; r < R; ++r) rstd[r] = 1.0f / sqrtf(rstd[r] * inv_c + a.eps);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r * groups + group;
      if (row >= a.rows) break;  // whole groups
      if (kOut == kOutY && t == 0) {
        if (a.mean) a.mean[row] = mean[r];
        if (a.rstd) a.rstd[row] = rstd[r];
      }
      if (!live) continue;  // whole quads / octets of lanes: items is a multiple of 4 / 8
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[r][h][i] = fmaf(x[r][h][i] * rstd[r], w[h][i], b[h][i]);
      store_item<T, kOut, kRows>(a, x[r], row, t, c, info);
    }
  }
}

// Backward. A workgroup walks rows blockIdx.x, + gridDim.x, ...; a thread owns
// the same kRuns runs of 8 columns in every row and keeps their weight and its
// part of dw and db in registers (with 4 or 8 runs, beyond 16384 columns, mostly in
// scratch memory). The parts of all workgroups go to `parts` ([gridDim.x][2][c]) and
// are added in a fixed order by the kernel below.
// Behind a row's last column x and dy are 0, and xhat = -mean rstd may overflow:
// infinity times 0 would make the whole row's mean(g xhat) a NaN. So the mean is 0
// there, or (where a run may be part of a row) x another element of the row.
// Bound: HBM, x and dy read and dx written once: 57600 x 5120 bf16 325 us (5.4 TB/s),
// 57600 x 13824 925 us (5.2 TB/s), 777 x 1003 fp32 8.2 us; but 4096 x 20480 504 us
// (1.0 TB/s) and 4096 x 65536 3.5 ms, by their scratch memory.
template <typename T, int kRuns, bool kSums, int kRows>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(NormBackArgs a) {
  __shared__ float sums[2][2][16];
  const int t = threadIdx.x, nt = blockDim.x, c = a.c;
  const int waves = nt >> 6;
  const float inv_c = 1.0f / (float)c;
  float w[kRuns][8], dw[kRuns][8], db[kRuns][8];
#pragma unroll
  for (int n = 0; n < kRuns; ++n) {
    load_w8<kRows>(a.w, a.w_bf16, (n * nt + t) * 8, c, 1.0f, w[n]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[n][i] = db[n][i] = 0.0f;
  }
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const T* xs = reinterpret_cast<const T*>(a.x) + row * a.ldx;
    const T* ds = reinterpret_cast<const T*>(a.dy) + row * a.lddy;
    Run8<T> xr[kRuns], dr[kRuns];
#pragma unroll
    for (int n = 0; n < kRuns; ++n) {
      const int col = (n * nt + t) * 8;
      xr[n].template load<kRows, kRows != kAligned>(xs, col, c);
      dr[n].template load<kRows>(ds, col, c);
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float mu[kRuns];  // kAligned: a run is whole or empty, the last one of a thread only
#pragma unroll
    for (int n = 0; n < kRuns; ++n)
      mu[n] = kRows == kAligned && n == kRuns - 1 && (n * nt + t) * 8 >= c ? 0.0f : mean;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int n = 0; n < kRuns; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xhat = (xr[n].get(i) - mu[n]) * rstd, d = dr[n].get(i);
        const float g = d * w[n][i];
        s1 += g;
        s2 = fmaf(g, xhat, s2);
        if constexpr (kSums) {
          dw[n][i] = fmaf(d, xhat, dw[n][i]);
          db[n][i] += d;
        }
      }
    // two slots in turn: a wave that is a row ahead writes the other one
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if ((t & 63) == 0) {
      sums[flip][0][t >> 6] = s1;
      sums[flip][1][t >> 6] = s2;
    }
    __syncthreads();
    s1 = row16_sum((t & 15) < waves ? sums[flip][0][t & 15] : 0.0f) * inv_c;
    s2 = row16_sum((t & 15) < waves ? sums[flip][1][t & 15] : 0.0f) * inv_c;
    T* o = reinterpret_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int n = 0; n < kRuns; ++n) {
      const int col = (n * nt + t) * 8;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xhat = (xr[n].get(i) - mu[n]) * rstd;
        v[i] = (dr[n].get(i) * w[n][i] - s1 - xhat * s2) * rstd;
      }
      store_run8<kRows>(o + col, c - col, v);
    }
  }
  if constexpr (kSums) {
    float* p = a.parts + (int64_t)blockIdx.x * 2 * c;
#pragma unroll
    for (int n = 0; n < kRuns; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = (n * nt + t) * 8 + i;
        if (col < c) {
          p[col] = dw[n][i];
          p[c + col] = db[n][i];
        }
      }
  }
}

// The same for rows of up to 256 columns: groups of kLanes = 16 or 32 lanes take a
// row each (above, a wave would have most lanes without a run, and a row a barrier).
// The groups' sums are added in order before they leave as the workgroup's part.
// Measured with the parts' sum, us, the kernel above and this one: 1000000 x 128 bf16
// 328 and 153 (5.0 TB/s), 500000 x 256 196 and 152, 23025 x 106 fp32 24.9 and 12.5,
// 1000 x 128 7.4 and 6.7, 77 x 200 8.3 and 8.8.
template <typename T, bool kSums, int kRows, int kLanes>
__global__ __launch_bounds__(256) void layer_norm_backward_narrow_kernel(NormBackArgs a) {
  constexpr int kGroups = 256 / kLanes, kCols = kLanes * 8;
  __shared__ float sums[kSums ? kGroups : 1][2][kCols];
  const int t = threadIdx.x & (kLanes - 1), group = threadIdx.x / kLanes, c = a.c, col = t * 8;
  const float inv_c = 1.0f / (float)c;
  float w[8], dw[8], db[8];
  load_w8<kRows>(a.w, a.w_bf16, col, c, 1.0f, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row0 = (int64_t)blockIdx.x * kGroups; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kGroups) {
    const bool live = row0 + group < a.rows;
    const int64_t row = live ? row0 + group : a.rows - 1;  // read again, not stored or summed
    Run8<T> xr, dr;
    xr.template load<kRows, true>(reinterpret_cast<const T*>(a.x) + row * a.ldx, col, c);
    dr.template load<kRows>(reinterpret_cast<const T*>(a.dy) + row * a.lddy, col, c);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xhat = (xr.get(i) - mean) * rstd, d = dr.get(i);
      const float g = d * w[i];
      s1 += g;
      s2 = fmaf(g, xhat, s2);
      if constexpr (kSums) {
        dw[i] = live ? fmaf(d, xhat, dw[i]) : dw[i];
        db[i] = live ? db[i] + d : db[i];
      }
    }
    s1 = lanes_sum<kLanes>(s1) * inv_c;
    s2 = lanes_sum<kLanes>(s2) * inv_c;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xhat = (xr.get(i) - mean) * rstd;
      v[i] = (dr.get(i) * w[i] - s1 - xhat * s2) * rstd;
    }
    if (live) store_run8<kRows>(reinterpret_cast<T*>(a.dx) + row * a.lddx + col, c - col, v);
  }
  if constexpr (kSums) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[group][0][col + i] = dw[i];
      sums[group][1][col + i] = db[i];
    }
    __syncthreads();
    float* p = a.parts + (int64_t)blockIdx.x * 2 * c;
    for (int j = threadIdx.x; j < 2 * c; j += 256) {
      const int which = j >= c, at = which ? j - c : j;
      float s = sums[0][which][at];
      for (int g = 1; g < kGroups; ++g) s += sums[g][which][at];
      p[j] = s;
    }
  }
}

// Sums the workgroups' parts: 32 columns a workgroup; its 32 half waves take the
// parts in turn, 8 loads in flight each, and their sums are added in order (512
// parts of 5120 columns 5.5 us).
__global__ __launch_bounds__(1024) void layer_norm_parts_kernel(const float* __restrict__ parts,
                                                                int n_parts, int c, void* dw,
                                                                void* db, bool w_bf16) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane, cols = 2 * (int64_t)c;
  const float* p = parts + min(col, cols - 1);
  float s = 0.0f;
  for (int p0 = half; p0 < n_parts; p0 += 8 * 32) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = p[min(p0 + u * 32, n_parts - 1) * cols];
#pragma unroll
    for (int u = 0; u < 8; ++u) s += p0 + u * 32 < n_parts ? v[u] : 0.0f;
  }
  sums[half][lane] = s;
  __syncthreads();
  if (half == 0 && col < cols) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) s += sums[w][lane];
    void* out = col < c ? dw : db;
    const int64_t i = col < c ? col : col - c;
    if (out) {
      if (w_bf16) reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)f32_to_bf16(s);
      else reinterpret_cast<float*>(out)[i] = s;
    }
  }
}

// Which forward kernel, by measurement on bf16 rows (us).
// Rows at once of layer_norm_rows_kernel, to the type itself unless named:
//   rows x columns     1      2      4
//   256 x 5120        7.5    7.5
//   512 x 13824      15.0   11.4
//   2048 x 5120      15.1   12.9   12.7
//   8192 x 5120        36     35     42
//   57600 x 1024       40     37     89
//   57600 x 5120      271    235    247
//   57600 x 13824     774    674    656
//   fp32 57600 x 5120 582    561    744
//   HiF4 57600 x 8192 348    323    403
// so two, from two rows a CU on. Rows that are not 16-byte aligned (5119 columns):
// bf16 292 and 267, fp32 641 and 759, so fp32 takes one there.
// Rows of up to 512 columns, a wave each and 8, 16 or 32 lanes each: bf16 2300000 x 128
// 650 and 254 (to HiF4 1289 and 191, to E4M3 885 and 184), 1000000 x 64 291 and 54,
// 500000 x 256 171 and 116, 200000 x 512 93 and 96 (to HiF4 126 and 71); 5000 x 128
// and fewer the same.
// A wave per row against it, into a quantizer: HiF4 57600 x 5120 215 and 315,
// 57600 x 6144 295 and 349, 2048 x 5120 12.5 and 17.8, 1024 x 5120 11.5 and 10.2;
// but 57600 x 4096 185 and 163, 57600 x 8192 486 and 323 (E4M3 the same way: 176 and
// 213, 226 and 258, 144 and 139, 329 and 286). At 57600 x 7168 the two outputs differ:
// HiF4 421 and 361, E4M3 253 and 272; so 5 and 6 waves for both. Workgroups of 5, 6
// and 7 waves leave the SIMDs of a CU unevenly filled, 4 and 8 do not; and a wave's own
// row needs more registers with every 1024 columns. More than 8 waves were not tried
// (weight and bias would leave 64 KB of LDS).
template <typename T, int kOut, int kRows>
static hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  const int items = kOut == kOutFp8 ? a.kp / 16 : (a.c + 15) / 16;
  const int waves = (items + 63) / 64;
#define HIF4_NORM(rr, multi, grid, waves, lanes)                                             \
  hipLaunchKernelGGL((layer_norm_rows_kernel<T, rr, kOut, multi, kRows, lanes>), dim3(grid), \
                     dim3(64 * (waves)), 0, stream, a)
  const auto narrow_grid = [&](int lanes) {  // workgroups of 4 waves
    const int64_t at_once = 256 / lanes;
    return (unsigned)std::min<int64_t>((a.rows + at_once - 1) / at_once, 256 * 16);
  };
  if constexpr (kRows == kTiny) {  // c < 8
    HIF4_NORM(1, false, narrow_grid(8), 4, 8);
    return hipGetLastError();
  } else {
    if (items <= 8) {
      HIF4_NORM(1, false, narrow_grid(8), 4, 8);
      return hipGetLastError();
    }
    if (items <= 16) {
      HIF4_NORM(1, false, narrow_grid(16), 4, 16);
      return hipGetLastError();
    }
    if (items <= 32) {
      HIF4_NORM(1, false, narrow_grid(32), 4, 32);
      return hipGetLastError();
    }
    if (items > 1024) {
      const unsigned grid = (unsigned)std::min<int64_t>(a.rows, 256 * 32);
      hipLaunchKernelGGL((layer_norm_wide_kernel<T, 4, kOut, kRows>), dim3(grid), dim3(1024), 0,
                         stream, a);
      return hipGetLastError();
    }
    if constexpr (sizeof(T) == 2 && kRows == kAligned && kOut != kOutY) {
      if ((waves == 5 || waves == 6) && a.rows >= 256 * 8) {
        const dim3 grid((unsigned)std::min<int64_t>((a.rows + 7) / 8, 256 * 8)), block(512);
        const size_t lds = (size_t)items * 8 * sizeof(float4);
        if (waves == 5)
          hipLaunchKernelGGL((layer_norm_wave_kernel<5, kOut>), grid, block, lds, stream, a);
        else
          hipLaunchKernelGGL((layer_norm_wave_kernel<6, kOut>), grid, block, lds, stream, a);
        return hipGetLastError();
      }
    }
    constexpr int kMany = kRows == kAligned || sizeof(T) == 2 ? 2 : 1;
    const int r = a.rows >= 256 * 2 ? kMany : 1;
    const unsigned grid =
        (unsigned)std::min<int64_t>((a.rows + r - 1) / r, (int64_t)256 * 64 / waves);
    if (r == kMany) {
      if (waves > 1) HIF4_NORM(kMany, true, grid, waves, 64);
      else HIF4_NORM(kMany, false, grid, 1, 64);
    } else {
      if (waves > 1) HIF4_NORM(1, true, grid, waves, 64);
      else HIF4_NORM(1, false, grid, 1, 64);
    }
    return hipGetLastError();
  }
#undef HIF4_NORM
}

// Runs of 8 columns a thread, and threads a workgroup, of the backward.
static int backward_runs(int64_t c) {
  const int64_t runs = (c + 7) / 8;
  return runs <= 512 ? 1 : runs <= 2048 ? 2 : runs <= 4096 ? 4 : 8;
}
static int backward_threads(int64_t c) {
  const int64_t runs = (c + 7) / 8, kr = backward_runs(c);
  return (int)(((runs + kr - 1) / kr + 63) / 64 * 64);
}

template <typename T, int kRows>
static hipError_t launch_norm_backward(const NormBackArgs& a, int grid, hipStream_t stream) {
  const int kr = backward_runs(a.c);
  const int threads = backward_threads(a.c);
#define HIF4_NARROW(lanes)                                                                         \
  do {                                                                                             \
    if (a.parts)                                                                                   \
      hipLaunchKernelGGL((layer_norm_backward_narrow_kernel<T, true, kRows, lanes>), dim3(grid),   \
                         dim3(256), 0, stream, a);                                                 \
    else                                                                                           \
      hipLaunchKernelGGL((layer_norm_backward_narrow_kernel<T, false, kRows, lanes>), dim3(grid),  \
                         dim3(256), 0, stream, a);                                                 \
    return hipGetLastError();                                                                      \
  } while (0)
  if (a.c <= 128) HIF4_NARROW(16);
  if constexpr (kRows != kTiny) {
    if (a.c <= 256) HIF4_NARROW(32);
  }
#undef HIF4_NARROW
#define HIF4_BACK(k)                                                                               \
  do {                                                                                             \
    if (a.parts)                                                                                   \
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, k, true, kRows>), dim3(grid), dim3(threads), 0,   \
                         stream, a);                                                               \
    else                                                                                           \
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, k, false, kRows>), dim3(grid), dim3(threads), 0,  \
                         stream, a);                                                               \
  } while (0)
  if constexpr (kRows != kTiny) {  // (c < 8 has returned)
    switch (kr) {
      case 1: HIF4_BACK(1); break;
      case 2: HIF4_BACK(2); break;
      case 4: HIF4_BACK(4); break;
      default: HIF4_BACK(8); break;
    }
  }
#undef HIF4_BACK
  return hipGetLastError();
}

}  // namespace hif4

using namespace hif4;

hipError_t hif4_launch_layer_norm(const NormArgs& a, bool x_bf16, int out, hipStream_t stream) {
  const auto go = [&](auto type, auto kind) {
    using T = decltype(type);
    constexpr int kOut = decltype(kind)::value;
    if (a.vec) return launch_norm<T, kOut, kAligned>(a, stream);
    if constexpr (kOut != kOutHif4) {  // (c % 64 == 0 there)
      if (a.c < 8) return launch_norm<T, kOut, kTiny>(a, stream);
    }
    return launch_norm<T, kOut, kAny>(a, stream);
  };
  const auto by_type = [&](auto kind) {
    return x_bf16 ? go(uint16_t{}, kind) : go(float{}, kind);
  };
  switch (out) {
    case kOutY: return by_type(std::integral_constant<int, kOutY>{});
    case kOutHif4: return by_type(std::integral_constant<int, kOutHif4>{});
    default: return by_type(std::integral_constant<int, kOutFp8>{});
  }
}

// Workgroups of the backward: up to 4096 columns 16 waves a CU, beyond two
// workgroups a CU. Measured (bf16, with the sums of the parts): 57600 x 1280, 3
// waves, 2 workgroups a CU 146 us, 5 95 us; 57600 x 5120, 5 waves of two runs, 2
// workgroups 330 us, 3 414 us.
// Fewer rows: the least k <= 8 with 64 k^2 >= rows each, which weighs a workgroup's
// rows in turn against the parts to be written and read again. Measured, us, at
// 1, 2, 3, 4 and 8 rows each: 100 x 1003 8.5, 8.0, 8.5, 9.6, 12.1; 777 x 1003 15.7,
// 11.7, 10.8, 10.1, 12.5; 1024 x 5120 28.4, 28.3, 25.2, 20.5, 21.2; 4096 x 1024
// 27.4, 27.4, 22.2, 18.3, 15.3.
int hif4_layer_norm_backward_parts(int64_t rows, int64_t c) {
  const int64_t at_once = c <= 128 ? 16 : c <= 256 ? 8 : 1;  // rows a workgroup has in hand
  const int64_t waves = c <= 256 ? 4 : backward_threads(c) / 64;
  const int64_t per_cu = backward_runs(c) == 1 ? std::max<int64_t>(2, 16 / waves) : 2;
  const int64_t turns = (std::max<int64_t>(rows, 1) + at_once - 1) / at_once;
  int64_t k = 1;
  while (k < 8 && 64 * k * k < turns) ++k;
  return (int)std::min<int64_t>((turns + k - 1) / k, 256 * per_cu);
}

hipError_t hif4_launch_layer_norm_backward(const NormBackArgs& a, bool x_bf16, void* dw, void* db,
                                           hipStream_t stream) {
  const int grid = hif4_layer_norm_backward_parts(a.rows, a.c);
  const auto by_type = [&](auto mode) {
    constexpr int kRows = decltype(mode)::value;
    return x_bf16 ? launch_norm_backward<uint16_t, kRows>(a, grid, stream)
                  : launch_norm_backward<float, kRows>(a, grid, stream);
  };
  const hipError_t e = a.vec      ? by_type(std::integral_constant<int, kAligned>{})
                       : a.c >= 8 ? by_type(std::integral_constant<int, kAny>{})
                                  : by_type(std::integral_constant<int, kTiny>{});
  if (e != hipSuccess || !a.parts) return e;
  hipLaunchKernelGGL(layer_norm_parts_kernel, dim3((unsigned)((2 * (int64_t)a.c + 31) / 32)),
                     dim3(1024), 0, stream, a.parts, grid, a.c, dw, db, a.w_bf16);
  return hipGetLastError();
}
