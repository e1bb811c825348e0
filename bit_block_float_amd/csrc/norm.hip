// norm.hip -- layer norm over the rows of a matrix: forward, forward that ends
// in a quantizer (HiF4 or E4M3 blocks), and backward with the reduction of the
// weight's and bias' gradients. HBM-streaming kernels for gfx950.
//
// Forward: y = (x - mean) rstd w + b with rstd = (var + eps)^(-1/2). A row is
// held in registers from its one read, so the variance is the mean of
// (x - mean)^2 over the same registers, not a difference of two large sums.
// Backward, with xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum over rows of dy xhat,  db = sum over rows of dy.
// Statistics, sums and gradients are fp32; results are rounded once.
#include <algorithm>

#include "fp8_dev.h"
#include "norm_dev.h"
#include "quant_dev.h"

namespace hif4 {

enum NormOut { kOutY = 0, kOutHif4 = 1, kOutFp8 = 2 };

// Sum over the lanes of a wave, the same bits in every lane (butterfly order).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sum over the P threads that share a row (P = 64: one wave; else the whole
// workgroup). `slot` is LDS of P / 64 floats that no other sum in flight uses.
template <int P>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if constexpr (P > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < P / 64; ++i) v += slot[i];
  }
  return v;
}

// 8 weights or biases from column `col` (fp32 or bf16), 1 / 0 without one.
__device__ __forceinline__ void load_w8(const void* w, bool w_bf16, bool vec, int col, int c,
                                        float fallback, float (&v)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fallback;
  } else if (w_bf16) {
    Run8<uint16_t> r;
    r.load(reinterpret_cast<const uint16_t*>(w) + col, c - col, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
  } else {
    Run8<float> r;
    r.load(reinterpret_cast<const float*>(w) + col, c - col, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
  }
}

__device__ __forceinline__ void store_run8(uint16_t* p, int valid, bool vec, const float (&v)[8]) {
  if (vec && valid >= 8) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                   f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint16_t)f32_to_bf16(v[i]);
  }
}
__device__ __forceinline__ void store_run8(float* p, int valid, bool vec, const float (&v)[8]) {
  if (vec && valid >= 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = v[i];
  }
}

// Forward. P threads share a row; a lane owns items (16 consecutive elements)
// t, t + P, ..., the quantizers' own mapping, so 4 aligned lanes hold a HiF4
// unit and 8 an E4M3 block when the row leaves through one of them. The value
// quantized is the one kOutY would store (rounded to bf16 for HiF4, to x's type
// for E4M3), so the codes are those of the two calls in turn.
template <typename T, int P, int kItems, int kOut>
__global__ __launch_bounds__(P > 64 ? P : 256) void layer_norm_kernel(NormArgs a) {
  constexpr int kRowsPerBlock = P > 64 ? 1 : 4;
  __shared__ float slots[2][P / 64];
  const int t = P > 64 ? threadIdx.x : (threadIdx.x & 63);
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
        uint32_t m16 = 0;
        if (j < items) {
          const uint4 mk = *reinterpret_cast<const uint4*>(a.mask + (size_t)j * 16);
          m16 = nonzero_bytes(mk.x) | (nonzero_bytes(mk.y) << 4) | (nonzero_bytes(mk.z) << 8) |
                (nonzero_bytes(mk.w) << 12);
        }
        const uint32_t cnt = __popc(m16);
        uint32_t incl = cnt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const uint32_t o = (uint32_t)__shfl_up((int)incl, d, 64);
          if ((t & 63) >= d) incl += o;
        }
        uint32_t base = run, total = (uint32_t)__shfl((int)incl, 63, 64);
        if constexpr (P > 64) {
          if ((t & 63) == 63) part[t >> 6] = incl;
          __syncthreads();
          total = 0;
          for (int w = 0; w < P / 64; ++w) {
            if (w < (t >> 6)) base += part[w];
            total += part[w];
          }
          __syncthreads();
        }
        info[n] = (m16 << 16) | ((base + incl - cnt) & 0xFFFFu);
        run += total;
      }
    }
  }

  const float inv_c = 1.0f / (float)c;
  const int64_t step = (int64_t)gridDim.x * kRowsPerBlock;
  for (int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + (P > 64 ? 0 : threadIdx.x >> 6);
       row < a.rows; row += step) {
    const T* src = x + row * a.ld;
    Run8<T> r0[kItems], r1[kItems];
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int col = (n * P + t) * 16;
      r0[n].load(src + col, c - col, a.vec);
      r1[n].load(src + col + 8, c - col - 8, a.vec);
    }
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < kItems; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += r0[n].get(i) + r1[n].get(i);
    const float mean = row_sum<P>(s, slots[0]) / (float)c;
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
    const float var = row_sum<P>(q, slots[1]) * inv_c;
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
        load_w8(a.w, a.w_bf16, a.w_vec, col + 8 * h, c, 1.0f, w);
        load_w8(a.b, a.w_bf16, a.w_vec, col + 8 * h, c, 0.0f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[h][i] = fmaf(((h ? r1[n] : r0[n]).get(i) - mean) * rstd, w[i], b[i]);
      }
      if constexpr (kOut == kOutY) {
        T* dst = reinterpret_cast<T*>(a.y) + row * a.ldy + col;
        store_run8(dst, c - col, a.y_vec, y[0]);
        store_run8(dst + 8, c - col - 8, a.y_vec, y[1]);
      } else if constexpr (kOut == kOutHif4) {
        uint32_t wds[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = y[i >> 2][2 * (i & 3)], hi = y[i >> 2][2 * (i & 3) + 1];
          wds[i] = f32x2_to_bf16x2(lo, hi);
        }
        uint4 v0 = make_uint4(wds[0], wds[1], wds[2], wds[3]);
        uint4 v1 = make_uint4(wds[4], wds[5], wds[6], wds[7]);
        if (a.mask) {
          keep_item_values(v0, v1, info[n], row, a.kept, a.n_mask);
          uint32_t z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t lo = (info[n] >> (16 + 2 * i)) & 1u, hi = (info[n] >> (17 + 2 * i)) & 1u;
            z[i] = ~((lo * 0x0000FFFFu) | (hi * 0xFFFF0000u));
          }
          v0 = make_uint4(v0.x & z[0], v0.y & z[1], v0.z & z[2], v0.w & z[3]);
          v1 = make_uint4(v1.x & z[4], v1.y & z[5], v1.z & z[6], v1.w & z[7]);
        }
        quantize_item(v0, v1, (uint32_t)j, (uint32_t)j,
                      reinterpret_cast<uint32_t*>(a.codes + row * (c / 2)), a.meta + row * (c / 64));
      } else {
        uint32_t am = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (sizeof(T) == 2) y[h][i] = bf16lo_to_f32(f32_to_bf16(y[h][i]));
            if (col + 8 * h + i >= c) y[h][i] = 0.0f;  // the padding of the last block
            am = max(am, abs_bits(y[h][i]));
          }
        const uint32_t e = e8m0_of(max8_u32(am));
        const float inv = e8m0_inv(min(e, 254u));
        uint4 w = make_uint4(encode4(y[0][0], y[0][1], y[0][2], y[0][3], inv),
                             encode4(y[0][4], y[0][5], y[0][6], y[0][7], inv),
                             encode4(y[1][0], y[1][1], y[1][2], y[1][3], inv),
                             encode4(y[1][4], y[1][5], y[1][6], y[1][7], inv));
        if (e == 255u) w = make_uint4(kFp8NaN4, kFp8NaN4, kFp8NaN4, kFp8NaN4);
        *reinterpret_cast<uint4*>(a.codes + row * a.kp + col) = w;
        if ((j & 7) == 0) a.scales[row * a.lds + (j >> 3)] = (uint8_t)e;
      }
    }
  }
}

// Backward. A workgroup walks rows blockIdx.x, + gridDim.x, ...; a thread owns
// the same kRuns runs of 8 columns in every row and keeps their weight and its
// part of dw and db in registers. The parts of all workgroups go to `parts`
// ([gridDim.x][2][c]) and are added in a fixed order by the kernel below.
template <typename T, int kRuns, bool kSums>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(NormBackArgs a) {
  __shared__ float sums[2][2][16];
  const int t = threadIdx.x, nt = blockDim.x, c = a.c;
  const int waves = nt >> 6;
  const float inv_c = 1.0f / (float)c;
  float w[kRuns][8], dw[kRuns][8], db[kRuns][8];
#pragma unroll
  for (int n = 0; n < kRuns; ++n) {
    load_w8(a.w, a.w_bf16, a.w_vec, (n * nt + t) * 8, c, 1.0f, w[n]);
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
      xr[n].load(xs + col, c - col, a.vec);
      dr[n].load(ds + col, c - col, a.vec);
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int n = 0; n < kRuns; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xhat = (xr[n].get(i) - mean) * rstd, d = dr[n].get(i);
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
    s1 = s2 = 0.0f;
    for (int i = 0; i < waves; ++i) {
      s1 += sums[flip][0][i];
      s2 += sums[flip][1][i];
    }
    s1 *= inv_c;
    s2 *= inv_c;
    T* o = reinterpret_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int n = 0; n < kRuns; ++n) {
      const int col = (n * nt + t) * 8;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xhat = (xr[n].get(i) - mean) * rstd;
        v[i] = (dr[n].get(i) * w[n][i] - s1 - xhat * s2) * rstd;
      }
      store_run8(o + col, c - col, a.dx_vec, v);
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

// Sums the workgroups' parts: 64 columns a workgroup, 16 runs of parts each
// added by one wave, the 16 sums added in order.
__global__ __launch_bounds__(1024) void layer_norm_parts_kernel(const float* __restrict__ parts,
                                                                int n_parts, int c, void* dw,
                                                                void* db, bool w_bf16) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (col < 2 * (int64_t)c)
    for (int p = wave; p < n_parts; p += 16) s += parts[(int64_t)p * 2 * c + col];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < 2 * (int64_t)c) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    void* out = col < c ? dw : db;
    const int64_t i = col < c ? col : col - c;
    if (out) {
      if (w_bf16) reinterpret_cast<uint16_t*>(out)[i] = (uint16_t)f32_to_bf16(s);
      else reinterpret_cast<float*>(out)[i] = s;
    }
  }
}

template <typename T, int kOut>
static hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  const int cols = kOut == kOutFp8 ? a.kp : (a.c + 15) / 16 * 16;
  const unsigned wave_grid = (unsigned)std::min<int64_t>((a.rows + 3) / 4, 256 * 32);
  const unsigned row_grid = (unsigned)std::min<int64_t>(a.rows, 256 * 32);
#define HIF4_NORM(P, items)                                                               \
  hipLaunchKernelGGL((layer_norm_kernel<T, P, items, kOut>), dim3(P > 64 ? row_grid : wave_grid), \
                     dim3(P > 64 ? P : 256), 0, stream, a)
  const bool wide = sizeof(T) == 4;
  if (cols <= 64 * 16) HIF4_NORM(64, 1);
  else if (cols <= 64 * 16 * 2) HIF4_NORM(64, 2);
  else if (!wide && cols <= 64 * 16 * 5) HIF4_NORM(64, 5);
  else if (cols <= 256 * 16 * 2) HIF4_NORM(256, 2);
  else if (cols <= 256 * 16 * 4) HIF4_NORM(256, 4);
  else HIF4_NORM(1024, 4);
#undef HIF4_NORM
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_norm_backward(const NormBackArgs& a, int grid, hipStream_t stream) {
  const int runs = (a.c + 7) / 8;
  const int per = (runs + 1023) / 1024 <= 1 ? (runs > 512 ? 2 : 1) : (runs + 1023) / 1024;
  const int kr = per <= 2 ? per : per <= 4 ? 4 : 8;
  const int threads = std::max(64, ((runs + kr - 1) / kr + 63) / 64 * 64);
#define HIF4_BACK(k)                                                                               \
  do {                                                                                             \
    if (a.parts)                                                                                   \
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, k, true>), dim3(grid), dim3(threads), 0,   \
                         stream, a);                                                               \
    else                                                                                           \
      hipLaunchKernelGGL((layer_norm_backward_kernel<T, k, false>), dim3(grid), dim3(threads), 0,  \
                         stream, a);                                                               \
  } while (0)
  switch (kr) {
    case 1: HIF4_BACK(1); break;
    case 2: HIF4_BACK(2); break;
    case 4: HIF4_BACK(4); break;
    default: HIF4_BACK(8); break;
  }
#undef HIF4_BACK
  return hipGetLastError();
}

}  // namespace hif4

using namespace hif4;

hipError_t hif4_launch_layer_norm(const NormArgs& a, bool x_bf16, int out, hipStream_t stream) {
  switch (out) {
    case kOutY:
      return x_bf16 ? launch_norm<uint16_t, kOutY>(a, stream) : launch_norm<float, kOutY>(a, stream);
    case kOutHif4:
      return x_bf16 ? launch_norm<uint16_t, kOutHif4>(a, stream)
                    : launch_norm<float, kOutHif4>(a, stream);
    default:
      return x_bf16 ? launch_norm<uint16_t, kOutFp8>(a, stream)
                    : launch_norm<float, kOutFp8>(a, stream);
  }
}

// Workgroups of the backward: two a CU, fewer for few rows.
int hif4_layer_norm_backward_parts(int64_t rows) {
  return (int)std::min<int64_t>(std::max<int64_t>(rows, 1), 512);
}

hipError_t hif4_launch_layer_norm_backward(const NormBackArgs& a, bool x_bf16, void* dw, void* db,
                                           hipStream_t stream) {
  const int grid = hif4_layer_norm_backward_parts(a.rows);
  hipError_t e = x_bf16 ? launch_norm_backward<uint16_t>(a, grid, stream)
                        : launch_norm_backward<float>(a, grid, stream);
  if (e != hipSuccess || !a.parts) return e;
  hipLaunchKernelGGL(layer_norm_parts_kernel, dim3((unsigned)((2 * (int64_t)a.c + 63) / 64)),
                     dim3(1024), 0, stream, a.parts, grid, a.c, dw, db, a.w_bf16);
  return hipGetLastError();
}
