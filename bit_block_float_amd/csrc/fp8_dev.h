// fp8_dev.h -- device helpers of the E4M3 block format (the rule is stated in
// hif4.h): the E8M0 scale of a block from its maximum, runs of 8 elements with
// guarded loads, and their encoding.
#pragma once

#include "hif4_dev.h"

namespace hif4 {

// Biased exponent (E8M0 byte) of the smallest power of two s >= 2^-127 with
// amax <= 448 s; `bits` = |amax| as fp32 bits. 448 = 1.75 * 2^8, so the
// exponent is that of amax minus 8, one more where the significand is above
// 1.75. 255 (E8M0's NaN) if the block holds a NaN or an infinity.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t bits) {
  const int e = (int)(bits >> 23) - 8 + (int)((bits & 0x7FFFFFu) > 0x600000u);
  return bits >= 0x7F800000u ? 255u : (uint32_t)max(e, 0);
}
// 2^(127 - byte), the reciprocal of the scale (byte <= 247 here: normal).
__device__ __forceinline__ float e8m0_inv(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// The scale itself; byte 0 is 2^-127 (subnormal in fp32), 255 is NaN.
__device__ __forceinline__ float e8m0_f32(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x400000u : byte << 23);
}

// Four E4M3 codes RNE(v * inv). v * inv is exact (a power of two, and no
// result leaves the normal fp32 range upwards), so the conversion's rounding
// is the only one.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}
constexpr uint32_t kFp8NaN4 = 0x7F7F7F7Fu;  // four E4M3 NaNs

// Four codes of two words of bf16 pairs: RNE(x / scale) by the scaled conversion
// (checked on every bf16 value against the rule over E8M0's range).
__device__ __forceinline__ uint32_t encode4_bf16(uint32_t lo, uint32_t hi, float scale) {
  typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
  typedef short half2_t __attribute__((ext_vector_type(2)));
  half2_t r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(pair_t, lo), scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(pair_t, hi), scale, true);
  return __builtin_bit_cast(uint32_t, r);
}

// How rows are read. Loads are unconditional, from clamped addresses (a load
// behind a branch is waited for at the branch's end, one after the other).
//  kAligned: rows are 16-byte aligned and c is a multiple of 8 (bf16) or 4 (fp32):
//    16-byte pieces, whole or empty.
//  kAny: c >= 8; the same loads at the elements' own alignment (global memory
//    takes any), the last pieces of a row moved back inside it and shifted.
//  kTiny: element by element.
enum RowAccess { kTiny = 0, kAny = 1, kAligned = 2 };

// m ? a : b by bits: a select may become a branch around the loads of its operands
__device__ __forceinline__ uint32_t pick(uint32_t m, uint32_t a, uint32_t b) {
  return (a & m) | (b & ~m);
}

// 8 consecutive elements of a row of c >= 1, from column col; elements at or past
// c are zero, or with kOther any other elements of the row.
template <typename T>
struct Run8;
template <>
struct Run8<uint16_t> {
  uint4 w;
  template <int kRows, bool kOther = false>
  __device__ __forceinline__ void load(const uint16_t* row, int col, int c) {
    if constexpr (kRows == kAligned) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + (col < c ? col : 0));
      const uint32_t m = kOther || col < c ? 0xFFFFFFFFu : 0u;
      w = make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
    } else if constexpr (kRows == kAny) {
      const int start = min(col, c - 8), skip = col - start;
      typedef uint32_t any4_t __attribute__((ext_vector_type(4), aligned(2)));
      const any4_t v = *reinterpret_cast<const any4_t*>(row + start);
      const uint32_t s4 = 0u - ((skip >> 2) & 1u), s2 = 0u - ((skip >> 1) & 1u);
      const uint32_t a0 = pick(s4, v[2], v[0]), a1 = pick(s4, v[3], v[1]);
      // shifted down by skip, or with kOther turned (what leaves comes in behind)
      const uint32_t a2 = pick(s4, kOther ? v[0] : 0u, v[2]);
      const uint32_t a3 = pick(s4, kOther ? v[1] : 0u, v[3]);
      const uint32_t b0 = pick(s2, a1, a0), b1 = pick(s2, a2, a1), b2 = pick(s2, a3, a2);
      const uint32_t b3 = pick(s2, kOther ? a0 : 0u, a3), sh = (skip & 1) * 16;
      const uint32_t m = kOther || skip < 8 ? 0xFFFFFFFFu : 0u;
      w = make_uint4(__builtin_amdgcn_alignbit(b1, b0, sh) & m,
                     __builtin_amdgcn_alignbit(b2, b1, sh) & m,
                     __builtin_amdgcn_alignbit(b3, b2, sh) & m,
                     __builtin_amdgcn_alignbit(kOther ? b0 : 0u, b3, sh) & m);
    } else {
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = row[min(col + i, c - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] &= kOther || col + i < c ? 0xFFFFu : 0u;
      w = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                     h[6] | (h[7] << 16));
    }
  }
  __device__ __forceinline__ void keep_if(bool ok) {
    const uint32_t m = ok ? 0xFFFFFFFFu : 0u;
    w = make_uint4(w.x & m, w.y & m, w.z & m, w.w & m);
  }
  // keeps the run as the words it was loaded as: the compiler cannot carry fp32
  // copies of the elements (twice the registers) past this point
  __device__ __forceinline__ void opaque() {
    asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
  }
  // the largest magnitude, as fp32 bits
  __device__ __forceinline__ uint32_t abs_max() const {
    // with the sign bits cleared, bf16 magnitudes order as integers (NaNs above infinity)
    const uint32_t m = pkmax_u16(pkmax_u16(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                pkmax_u16(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  // the 8 codes under the scale byte e (all NaN for 255)
  __device__ __forceinline__ uint2 encode(uint32_t e) const {
    const float s = e8m0_f32(e);
    const uint2 r = make_uint2(encode4_bf16(w.x, w.y, s), encode4_bf16(w.z, w.w, s));
    return e == 255u ? make_uint2(kFp8NaN4, kFp8NaN4) : r;
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t u = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
    return (i & 1) ? bf16hi_to_f32(u) : bf16lo_to_f32(u);
  }
};
template <>
struct Run8<float> {
  float v[8];
  template <int kRows, bool kOther = false>
  __device__ __forceinline__ void load(const float* row, int col, int c) {
    if constexpr (kRows == kAligned) {
      const float4 a = *reinterpret_cast<const float4*>(row + (col < c ? col : 0));
      const float4 b = *reinterpret_cast<const float4*>(row + (col + 4 < c ? col + 4 : 0));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = kOther || col + (i & 4) < c ? v[i] : 0.0f;
    } else if constexpr (kRows == kAny) {
      typedef uint32_t any4_t __attribute__((ext_vector_type(4), aligned(4)));
      any4_t q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q[h] = *reinterpret_cast<const any4_t*>(row + min(col + 4 * h, c - 4));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int skip = col + 4 * h - min(col + 4 * h, c - 4);
        const uint32_t s2 = 0u - ((skip >> 1) & 1u), s1 = 0u - (skip & 1u);
        const uint32_t m = kOther || skip < 4 ? 0xFFFFFFFFu : 0u;
        const uint32_t a0 = pick(s2, q[h][2], q[h][0]), a1 = pick(s2, q[h][3], q[h][1]);
        const uint32_t a2 = pick(s2, kOther ? q[h][0] : 0u, q[h][2]);
        const uint32_t a3 = pick(s2, kOther ? q[h][1] : 0u, q[h][3]);
        v[4 * h] = __uint_as_float(pick(s1, a1, a0) & m);
        v[4 * h + 1] = __uint_as_float(pick(s1, a2, a1) & m);
        v[4 * h + 2] = __uint_as_float(pick(s1, a3, a2) & m);
        v[4 * h + 3] = __uint_as_float(pick(s1, kOther ? a0 : 0u, a3) & m);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = row[min(col + i, c - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float(__float_as_uint(v[i]) & (kOther || col + i < c ? 0xFFFFFFFFu : 0u));
    }
  }
  __device__ __forceinline__ void keep_if(bool ok) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ok ? v[i] : 0.0f;
  }
  __device__ __forceinline__ uint32_t abs_max() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint2 encode(uint32_t e) const {
    const float inv = e8m0_inv(min(e, 254u));
    const uint2 r = make_uint2(encode4(v[0], v[1], v[2], v[3], inv),
                               encode4(v[4], v[5], v[6], v[7], inv));
    return e == 255u ? make_uint2(kFp8NaN4, kFp8NaN4) : r;
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
};

// Columns of 8 runs (8 rows x 8 columns): the largest magnitude of each column as
// fp32 bits, and the 8 codes of column i.
__device__ __forceinline__ void column_max(const Run8<uint16_t> (&v)[8], uint32_t (&m)[8]) {
  uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    p[0] = pkmax_u16(p[0], v[r].w.x & 0x7FFF7FFFu);
    p[1] = pkmax_u16(p[1], v[r].w.y & 0x7FFF7FFFu);
    p[2] = pkmax_u16(p[2], v[r].w.z & 0x7FFF7FFFu);
    p[3] = pkmax_u16(p[3], v[r].w.w & 0x7FFF7FFFu);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = (i & 1) ? p[i >> 1] & 0xFFFF0000u : p[i >> 1] << 16;
}
__device__ __forceinline__ void column_max(const Run8<float> (&v)[8], uint32_t (&m)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) m[i] = max(m[i], __float_as_uint(v[r].v[i]) & 0x7FFFFFFFu);
  }
}
__device__ __forceinline__ uint2 encode_column(const Run8<uint16_t> (&v)[8], int i, uint32_t e) {
  const float s = e8m0_f32(e);
  uint32_t p[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // rows 2q, 2q + 1 of the column as one word
    const uint4 &a = v[2 * q].w, &b = v[2 * q + 1].w;
    const uint32_t x = i < 2 ? a.x : i < 4 ? a.y : i < 6 ? a.z : a.w;
    const uint32_t y = i < 2 ? b.x : i < 4 ? b.y : i < 6 ? b.z : b.w;
    p[q] = __builtin_amdgcn_perm(y, x, (i & 1) ? 0x07060302u : 0x05040100u);
  }
  const uint2 r = make_uint2(encode4_bf16(p[0], p[1], s), encode4_bf16(p[2], p[3], s));
  return e == 255u ? make_uint2(kFp8NaN4, kFp8NaN4) : r;
}
__device__ __forceinline__ uint2 encode_column(const Run8<float> (&v)[8], int i, uint32_t e) {
  const float inv = e8m0_inv(min(e, 254u));
  const uint2 r = make_uint2(encode4(v[0].v[i], v[1].v[i], v[2].v[i], v[3].v[i], inv),
                             encode4(v[4].v[i], v[5].v[i], v[6].v[i], v[7].v[i], inv));
  return e == 255u ? make_uint2(kFp8NaN4, kFp8NaN4) : r;
}

}  // namespace hif4

// Internal (hidden) host launchers; argument checks happen in api_fp8.hip.
hipError_t hif4_launch_quantize_fp8(const void* x, bool bf16, int64_t rows, int64_t k, int64_t ld,
                                    int block_rows, uint8_t* codes, uint8_t* scales, int64_t lds,
                                    uint8_t* codes_t, uint8_t* scales_t, int64_t lds_t,
                                    hipStream_t stream);
hipError_t hif4_launch_dequantize_fp8(const uint8_t* codes, const void* scales, bool scales_f32,
                                      int block_rows, int64_t lds, int64_t rows, int64_t k,
                                      void* out, bool out_bf16, hipStream_t stream);
size_t hif4_gemm_fp8_ws_bytes(int64_t m, int64_t n, int64_t k);
// A product Y = X W^T (sizes above 0).
struct Fp8Product {
  const uint8_t *x, *xs;
  int64_t ldxs;
  const uint8_t* w;
  const void* ws;
  int64_t ldws;
  bool ws_f32;
  int w_block;
  int64_t m, n, k;
  void* y;
  bool y_bf16;
};
hipError_t hif4_launch_gemm_fp8(const Fp8Product& p, void* workspace, hipStream_t stream);
hipError_t hif4_launch_gemm_fp8_two(const Fp8Product& a, const Fp8Product& b, void* workspace,
                                    hipStream_t stream);
