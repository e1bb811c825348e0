// mxfp4_dev.h -- device helpers of the 4-bit microscaled format (MXFP4: E2M1
// elements, one E8M0 scale per 32; the rule is stated in hif4.h) and of groups of
// rows, and the internal launchers.
#pragma once

#include "fp8_dev.h"

namespace hif4 {

// Biased exponent (E8M0 byte) of the smallest power of two s >= 2^-127 with
// amax <= 6 s; `bits` = |amax| as fp32 bits. 6 = 1.5 * 2^2, so the exponent is
// that of amax minus 2, one more where the significand is above 1.5. 255 (E8M0's
// NaN) if the block holds a NaN or an infinity.
__device__ __forceinline__ uint32_t mx4_scale_of(uint32_t bits) {
  const uint32_t e = max((bits + 0x3FFFFFu) >> 23, 2u) - 2u;  // (carries above 1.5)
  return bits >= 0x7F800000u ? 255u : e;
}
// The scale of a byte below 255 (byte 0 is 2^-127, subnormal in fp32).
__device__ __forceinline__ float mx4_scale(uint32_t e) {
  return __uint_as_float(max(e << 23, 0x400000u));
}

constexpr uint32_t kMx4Nan8 = 0x77777777u;  // the codes of a block whose scale is NaN

// Two values to a byte of two codes, RNE(x / scale): byte kByte of `old`. The scaled
// conversion divides exactly and rounds once (checked on every bf16 value, and on
// fp32 ones between them, for scale bytes 0 to 253).
template <int kByte>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t old, uint32_t bf16x2, float scale) {
  typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(pair_t, bf16x2), scale, kByte);
}
template <int kByte>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, kByte);
}

// The 8 codes of a run under the scale byte e: element i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t mx4_encode(const Run8<uint16_t>& v, uint32_t e) {
  const float s = mx4_scale(e);
  uint32_t r = mx4_pair<0>(0u, v.w.x, s);
  r = mx4_pair<1>(r, v.w.y, s);
  r = mx4_pair<2>(r, v.w.z, s);
  r = mx4_pair<3>(r, v.w.w, s);
  return e == 255u ? kMx4Nan8 : r;
}
__device__ __forceinline__ uint32_t mx4_encode(const Run8<float>& v, uint32_t e) {
  const float s = mx4_scale(e);
  uint32_t r = mx4_pair<0>(0u, v.v[0], v.v[1], s);
  r = mx4_pair<1>(r, v.v[2], v.v[3], s);
  r = mx4_pair<2>(r, v.v[4], v.v[5], s);
  r = mx4_pair<3>(r, v.v[6], v.v[7], s);
  return e == 255u ? kMx4Nan8 : r;
}
// The 8 codes of column i of 8 runs (8 rows x 8 columns).
__device__ __forceinline__ uint32_t mx4_encode_column(const Run8<uint16_t> (&v)[8], int i, uint32_t e) {
  Run8<uint16_t> c;
  uint32_t p[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // rows 2q, 2q + 1 of the column as one word
    const uint4 &a = v[2 * q].w, &b = v[2 * q + 1].w;
    const uint32_t x = i < 2 ? a.x : i < 4 ? a.y : i < 6 ? a.z : a.w;
    const uint32_t y = i < 2 ? b.x : i < 4 ? b.y : i < 6 ? b.z : b.w;
    p[q] = __builtin_amdgcn_perm(y, x, (i & 1) ? 0x07060302u : 0x05040100u);
  }
  c.w = make_uint4(p[0], p[1], p[2], p[3]);
  return mx4_encode(c, e);
}
__device__ __forceinline__ uint32_t mx4_encode_column(const Run8<float> (&v)[8], int i, uint32_t e) {
  Run8<float> c;
#pragma unroll
  for (int r = 0; r < 8; ++r) c.v[r] = v[r].v[i];
  return mx4_encode(c, e);
}

// 8 elements that are all there, at an address aligned to 16 bytes (kAligned) or to the
// element.
template <int kRows>
__device__ __forceinline__ void load_whole(Run8<uint16_t>& r, const uint16_t* p) {
  if constexpr (kRows == kAligned) r.w = *reinterpret_cast<const uint4*>(p);
  else __builtin_memcpy(&r.w, p, 16);
}
template <int kRows>
__device__ __forceinline__ void load_whole(Run8<float>& r, const float* p) {
  if constexpr (kRows == kAligned) p = reinterpret_cast<const float*>(__builtin_assume_aligned(p, 16));
  __builtin_memcpy(r.v, p, 32);
}

// ---------------------------------------------------------------- groups of rows
//
// Group e is rows offsets[e] .. offsets[e + 1] - 1. What the offsets say is taken
// within the matrix (0 .. rows) and a group that would end before it begins as
// empty, so no offsets lead out of bounds.
struct Groups {
  const int64_t* offsets;  // on the device, [count + 1]; NULL: one group of all rows
  int count;
  int64_t rows;
};
__device__ __forceinline__ void group_range(const Groups& g, int e, int64_t& begin, int64_t& end) {
  begin = min(max(g.offsets[e], (int64_t)0), g.rows);
  end = max(begin, min(max(g.offsets[e + 1], (int64_t)0), g.rows));
}

// Rows are cut into units (tiles) of 2^shift, no unit reaching into two groups.
// group_units: how many there are in all; group_unit: the group of unit t, and the
// units before that group (false: there is no unit t); units_before: the units before
// group e. Every lane of the wave takes part, and each has the same result.
__device__ __forceinline__ uint32_t lanes_inclusive(uint32_t v) {
  // DPP moves: within rows of 16 lanes, then row 0's sum to row 1 and 2's to 3, then
  // the lower half's to the upper one
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);  // row_shr 1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);  // row_shr 2
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);  // row_shr 4
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);  // row_shr 8
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);  // row_bcast 15
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);  // row_bcast 31
  return v;
}
__device__ __forceinline__ uint32_t units_of(const Groups& g, int e, int shift) {
  int64_t begin, end;
  group_range(g, e, begin, end);
  return (uint32_t)((end - begin + (1 << shift) - 1) >> shift);
}
// (256 groups at a time: the loads of their offsets are in flight together)
struct Units4 {
  uint32_t n[4];
  __device__ __forceinline__ Units4(const Groups& g, int e0, int count, int shift) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = e0 + c * 64 + (int)(threadIdx.x & 63);
      n[c] = units_of(g, min(e, g.count - 1), shift);  // unconditional loads
      n[c] = e < count ? n[c] : 0u;
    }
  }
};
__device__ __forceinline__ uint32_t units_before(const Groups& g, int shift, int group) {
  uint32_t sum = 0;
  for (int e0 = 0; e0 < group; e0 += 256) {
    const Units4 u(g, e0, group, shift);
    sum += u.n[0] + u.n[1] + u.n[2] + u.n[3];
  }
  return (uint32_t)__builtin_amdgcn_readlane((int)lanes_inclusive(sum), 63);
}
__device__ __forceinline__ uint32_t group_units(const Groups& g, int shift) {
  return units_before(g, shift, g.count);
}
__device__ __forceinline__ bool group_unit(const Groups& g, int shift, uint32_t t, int& group,
                                           uint32_t& before) {
  uint32_t sum = 0;
  for (int e0 = 0; e0 < g.count; e0 += 256) {
    const Units4 u(g, e0, g.count, shift);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t incl = sum + lanes_inclusive(u.n[c]);
      const uint64_t past = __ballot(incl > t);
      if (past != 0) {
        const int first = __ffsll((unsigned long long)past) - 1;
        group = e0 + c * 64 + first;
        before = (uint32_t)__builtin_amdgcn_readlane((int)(incl - u.n[c]), first);
        return before <= t;  // (more only where offsets that do not ascend overflow the sum)
      }
      sum = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
    }
  }
  return false;
}

// Units of 2^shift rows that groups of as many rows can have at most.
inline int64_t most_units(int64_t rows, int64_t groups, int shift) {
  return (rows + (((int64_t)1 << shift) - 1) * groups) >> shift;
}

}  // namespace hif4

// Internal (hidden) host launchers; argument checks happen in api_mxfp4.hip.
// x: `batch` matrices [rows][ld]. codes, scales along the rows, codes_t, scales_t of
// the transpose (either pair may be NULL); offsets: groups of x's rows (batch 1).
hipError_t hif4_launch_quantize_mxfp4(const void* x, bool bf16, int64_t batch, int64_t rows, int64_t k,
                                      int64_t ld, const hif4::Groups& groups, uint8_t* codes,
                                      uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                                      hipStream_t stream);
hipError_t hif4_launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                        int64_t k, void* out, bool out_bf16, hipStream_t stream);

// A product Y = X W^T (sizes above 0), codes rows of ldx and ldw bytes, scale rows a
// 16th of that.
//  kMx4Plain   X [m], W [n], k / 128 runs of 128 along K.
//  kMx4Rows    X's rows are in groups, group e has W [n] number e.
//  kMx4Depth   K is in groups (of `groups.rows` values in all, group e's a run of
//              whole 128s at the 128s of those before it); Y [m][n] number e is group
//              e's sum.
enum Mx4Mode { kMx4Plain = 0, kMx4Rows = 1, kMx4Depth = 2 };
struct Mx4Product {
  const uint8_t *x, *xs;
  int64_t ldx;
  const uint8_t *w, *ws;
  int64_t ldw;
  int64_t m, n, k;  // k: kMx4Depth: all of a row (ldx * 2)
  void* y;
  bool y_bf16;
  int mode;
  hif4::Groups groups;
};
size_t hif4_gemm_mxfp4_ws_bytes(int64_t m, int64_t n, int64_t k);
hipError_t hif4_launch_gemm_mxfp4(const Mx4Product& p, void* workspace, hipStream_t stream);
hipError_t hif4_launch_gemm_mxfp4_two(const Mx4Product& a, const Mx4Product& b, void* workspace,
                                      hipStream_t stream);
