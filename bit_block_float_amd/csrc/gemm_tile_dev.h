// gemm_tile_dev.h -- what the tile kernels of the 8-bit and the 4-bit products
// share: direct-to-LDS loads, the way of a wave's results to memory, and the order
// of the tiles.
#pragma once

#include "hif4_dev.h"

namespace hif4 {

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(4))) uint32_t gu32x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t gu32x2_t;
typedef __attribute__((ext_vector_type(16))) float gf32x16_t;
typedef __attribute__((ext_vector_type(4))) float gf32x4_t;
typedef __attribute__((address_space(3))) void glds_void_t;

constexpr int kRsrc3 = 0x00020000;

// Direct-to-LDS loads of 16 (4) bytes a lane, to `dst` + 16 (4) * lane.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (glds_void_t*)dst, 16, voff, off, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (glds_void_t*)dst, 4, voff, off, 0, 0);
}

// Four consecutive columns of one row of Y.
template <bool kBf16>
__device__ __forceinline__ void store4(void* y, int64_t off, int col, int n, bool vec, float a,
                                       float b, float c, float d) {
  if constexpr (kBf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + off;
    if (vec && col + 4 <= n) {
      *reinterpret_cast<uint2*>(p) = make_uint2(f32x2_to_bf16x2(a, b), f32x2_to_bf16x2(c, d));
    } else {
      if (col < n) p[0] = (uint16_t)f32_to_bf16(a);
      if (col + 1 < n) p[1] = (uint16_t)f32_to_bf16(b);
      if (col + 2 < n) p[2] = (uint16_t)f32_to_bf16(c);
      if (col + 3 < n) p[3] = (uint16_t)f32_to_bf16(d);
    }
  } else {
    float* p = reinterpret_cast<float*>(y) + off;
    if (vec && col + 4 <= n) {
      *reinterpret_cast<gf32x4_t*>(p) = gf32x4_t{a, b, c, d};
    } else {
      if (col < n) p[0] = a;
      if (col + 1 < n) p[1] = b;
      if (col + 2 < n) p[2] = c;
      if (col + 3 < n) p[3] = d;
    }
  }
}

// The wave's part of Y: kTN x kTM blocks of 32 x 32 (block (i, j): columns from
// col0 + 32 i, rows from row0 + 32 j). In the MFMA's result lane l holds row
// l & 31 and, in group g of 4 registers, columns 8 g + 4 (l >> 5) .. + 3: stored
// from there, an instruction would touch 32 lines for 16 or 32 bytes each. The
// rows go through LDS instead (`stage`: the wave's own kStageBytes; a wave's LDS
// accesses complete in order) and leave as whole lines, past the caches' care
// (Y is read by no one here). Measured on 57600 x 13824 x 5120 with bf16 Y when
// the kernel took 3.85 ms: direct stores were 0.69 of it.
template <bool kBf16, int kTN>
constexpr int kStageBytes = 32 * (kTN * 32 * (kBf16 ? 2 : 4) + 16);

template <bool kBf16, int kTN, int kTM>
__device__ __forceinline__ void store_tile(gf32x16_t (&acc)[kTN][kTM], char* stage, void* Y,
                                           int64_t row0, int64_t col0, int64_t M, int64_t N,
                                           int lane) {
  constexpr int kE = kBf16 ? 2 : 4, kPer = 16 / kE;          // elements a 16-byte piece
  constexpr int kPitch = kTN * 32 * kE + 16;                 // rows start 4 banks apart
  constexpr int kLanes = kTN * 32 * kE / 16;                 // pieces a row
  constexpr int kRows = 64 / kLanes;                         // rows an instruction
  const bool vec = (N & (kPer - 1)) == 0 && ((uintptr_t)Y & 15) == 0;
  char* const put = stage + (lane & 31) * kPitch + (lane >> 5) * 4 * kE;
  const char* const get = stage + (lane / kLanes) * kPitch + (lane % kLanes) * 16;
  const int64_t row = row0 + lane / kLanes, col = col0 + (lane % kLanes) * kPer;
  const int rows = (int)max((int64_t)0, min(M - row, (int64_t)32 * kTM));  // from this lane's first on
  char* dst = reinterpret_cast<char*>(Y) + (row * N + col) * kE;
  const int64_t step = kRows * N * kE;
#pragma unroll
  for (int j = 0; j < kTM; ++j) {
    // 256 sums fill the accumulation registers: they stay there until their turn. (Copied
    // ahead of the branches they spilled: 57600 x 13824 x 5120 in MXFP4 3.6% slower, the bf16
    // weight gradients of 16 experts, 2048 x 5120 from 1024 rows each, 180 us instead of 162.)
    if constexpr (kTN * kTM == 16) {
#pragma unroll
      for (int i = 0; i < kTN; ++i) asm volatile("" : "+a"(acc[i][j]));
    }
#pragma unroll
    for (int i = 0; i < kTN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const gf32x16_t& a = acc[i][j];
        char* to = put + (i * 32 + 8 * g) * kE;
        if constexpr (kBf16)
          *reinterpret_cast<gu32x2_t*>(to) =
              gu32x2_t{f32x2_to_bf16x2(a[4 * g], a[4 * g + 1]),
                       f32x2_to_bf16x2(a[4 * g + 2], a[4 * g + 3])};
        else
          *reinterpret_cast<gf32x4_t*>(to) =
              gf32x4_t{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
      }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    const auto piece = [&](int p) { return *reinterpret_cast<const gu32x4_t*>(get + p * kRows * kPitch); };
    const auto has = [&](int p) { return j * 32 + p * kRows < rows; };
    if (col0 + 32 * kTN > N) {  // the last columns; rolled up, or this were most of the kernel's code
#pragma unroll 1
      for (int p = 0; p < 32 / kRows; ++p, dst += step) {
        const gu32x4_t v = piece(p);
        if (!has(p)) continue;
        if (col + kPer <= N) {
          __builtin_memcpy(dst, &v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            if (col + e >= N) break;
            if constexpr (kBf16)
              reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            else
              reinterpret_cast<uint32_t*>(dst)[e] = v[e];
          }
        }
      }
    } else if (vec && row0 + 32 * kTM <= M) {  // whole: no branch a store, which would wait for its read alone
      // (57600 x 13824 x 5120, bf16 Y: in E4M3 3009 us without this case, 2989 with it; in MXFP4 1945, 1928)
#pragma unroll
      for (int p = 0; p < 32 / kRows; ++p, dst += step)
        __builtin_nontemporal_store(piece(p), reinterpret_cast<gu32x4_t*>(dst));
    } else if (vec) {
#pragma unroll
      for (int p = 0; p < 32 / kRows; ++p, dst += step) {
        const gu32x4_t v = piece(p);
        if (has(p)) __builtin_nontemporal_store(v, reinterpret_cast<gu32x4_t*>(dst));
      }
    } else {  // rows of any alignment: whole pieces all the same
#pragma unroll
      for (int p = 0; p < 32 / kRows; ++p, dst += step) {
        const gu32x4_t v = piece(p);
        if (has(p)) __builtin_memcpy(dst, &v, 16);
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
}

// Tile (row, column) number t of tiles_m x tiles_n: column by column in groups of 4
// tile rows (57600 x 13824 x 5120 in E4M3: 3.03 ms; groups of 8 3.05, of 16 3.17).
__device__ __forceinline__ void tile_in(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, int64_t& tm,
                                        int64_t& tn) {
  const uint32_t group = 4, per_group = group * tiles_n;
  const uint32_t gi = t / per_group, first = gi * group, in = t - gi * per_group;
  const uint32_t gsize = min(tiles_m - first, group);
  tm = __builtin_amdgcn_readfirstlane(first + in % gsize);
  tn = __builtin_amdgcn_readfirstlane(in / gsize);
}

// Workgroup t's number among `total` tiles: consecutive workgroup ids go to different
// XCDs; each XCD gets a contiguous run of tiles.
__device__ __forceinline__ uint32_t xcd_order(uint32_t t, uint32_t total) {
  const uint32_t per_xcd = total / 8;
  return t < per_xcd * 8 ? (t & 7) * per_xcd + (t >> 3) : t;
}

__device__ __forceinline__ void tile_of(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, int64_t& tm,
                                        int64_t& tn) {
  tile_in(xcd_order(t, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
}

}  // namespace hif4
