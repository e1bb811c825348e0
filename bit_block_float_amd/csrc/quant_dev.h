// quant_dev.h -- the HiF4 encoder of one 16-element item (device code), used by
// the quantize kernels (quant.hip) and by the layer norm that quantizes its
// result (norm.hip). The rule is stated in hif4.h, the lane mapping in
// quant.hip.
#pragma once

#include "hif4_dev.h"

namespace hif4 {

// Max over the 4 lanes of an aligned quad (DPP quad_perm), and OR.
__device__ __forceinline__ uint32_t max4_u32(uint32_t v) {
  v = max(v, dpp<kDppQuadXor1>(v));
  v = max(v, dpp<kDppQuadXor2>(v));
  return v;
}
__device__ __forceinline__ uint32_t or4_u32(uint32_t v) {
  v |= dpp<kDppQuadXor1>(v);
  v |= dpp<kDppQuadXor2>(v);
  return v;
}

// ---- packed 16-bit element arithmetic
//
// The element step works on two bf16 values per 32-bit word with packed
// 16-bit instructions. For a level-3 quad with exponent sum E under a unit of
// code c (e = c >> 2, m = c & 3), the S1P2 magnitude is k = min(RNE(t), 7)
// with t = 4|x| / D = y * 4/(4+m), y = |x| 2^(33-e-E). Below range
// saturation every y lies under 7 * 1.75 (the level-3 rule bounds the quad
// maximum by 1.75 s 2^E), and any y of 16 or more gives k = 7, so y capped
// at 16 is an fp16 number: its bf16 bits become fp16 bits by one saturating
// subtract of ((e + E + 79) << 7) (exponent rebias and 2^(33-e-E) together;
// values too small for an fp16 normal saturate to 0 or land among the fp16
// subnormals, all of which round to k = 0) and a shift left by 3. Then
// t = fma(y, hi, y lo) in fp16, with hi = RN16(4/(4+m)) and
// lo = RN16(4/(4+m) - hi): within 2^-19 of the real quotient, while a
// non-tie quotient is at least 9 fp16 half-ulps from the nearest half-integer
// and a tie is an fp16 number, so t rounds on the same side as the real
// quotient and ties come out exact. Adding 1024 (fp16 spacing 1 there)
// rounds to nearest even; min(., 1031) saturates k at 7 and leaves k in the
// low byte of each half. (Checked on the CPU for every bf16 y below 14 and
// every m, and by the element-rounding parity tests.)
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t kpair(uint32_t absw, uint32_t csub, uint32_t hi2,
                                          uint32_t lo2) {
  u16x2_t y = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2_t, absw),
                                            __builtin_bit_cast(u16x2_t, csub));
  // range saturation (c = 255 below a unit maximum above 7 v(255)) lets y
  // exceed the fp16 range: cap it at 16 (pattern 0x0980 before the shift),
  // which still rounds to k = 7
  y = __builtin_elementwise_min(y, (u16x2_t)(0x0980));
  y = y << (u16x2_t)(3);
  const f16x2_t yf = __builtin_bit_cast(f16x2_t, y);
  const f16x2_t pl = yf * __builtin_bit_cast(f16x2_t, lo2);
  f16x2_t t = __builtin_elementwise_fma(yf, __builtin_bit_cast(f16x2_t, hi2), pl);
  t = t + (f16x2_t)((_Float16)1024.0f);
  t = __builtin_elementwise_min(t, (f16x2_t)((_Float16)1031.0f));
  return __builtin_bit_cast(uint32_t, t);  // k in bytes 0 and 2
}

// Larger of the two u16 halves.
__device__ __forceinline__ uint32_t hmax_u16(uint32_t v) { return max(v & 0xFFFFu, v >> 16); }

// RN16(4/(4+m)) and the fp16 remainder, both halves.
__device__ __forceinline__ uint32_t kinv_hi2(uint32_t m) {
  return select4(m, 0x3C003C00u, 0x3A663A66u, 0x39553955u, 0x38923892u);
}
__device__ __forceinline__ uint32_t kinv_lo2(uint32_t m) {
  return select4(m, 0x00000000u, 0x0A660A66u, 0x09550955u, 0x08920892u);
}

// Level-3 quad maxima of a level-2 group, as |x| bf16 bits: `a` = the group's
// 4 words with the sign bits cleared.
struct QuadMax {
  uint32_t a, b;
};
__device__ __forceinline__ QuadMax quad_max(uint4 a) {
  return QuadMax{hmax_u16(pkmax_u16(a.x, a.y)), hmax_u16(pkmax_u16(a.z, a.w))};
}

// One level-2 group (8 elements, one code word): steps 3-5 given the unit's
// level-1 code. w: the group's 8 bf16 values (element 2i in the low half of
// word i), a: the same with the sign bits cleared, qm: its quad maxima;
// thr2 / thr175: bf16 bits of 3.5 s and 1.75 s (exact: s has at most three
// significant bits). Returns the code word; e2 and e3 bits by reference.
__device__ __forceinline__ uint32_t encode_group(uint4 w, uint4 a, QuadMax qm, uint32_t e,
                                                 uint32_t hi2, uint32_t lo2, uint32_t thr2,
                                                 uint32_t thr175, uint32_t& e2, uint32_t& e3a,
                                                 uint32_t& e3b) {
  // steps 3-4: level-2 / level-3 bits (exact compares of bf16 bit patterns)
  e2 = max(qm.a, qm.b) > thr2;
  const uint32_t t3 = e2 ? thr2 : thr175;
  e3a = qm.a > t3;
  e3b = qm.b > t3;
  // step 5: k = RNE(4|x| / D), two elements per packed operation
  const uint32_t ca = ((e + e2 + e3a + 79u) << 7) * 0x00010001u;
  const uint32_t cb = ((e + e2 + e3b + 79u) << 7) * 0x00010001u;
  const uint32_t k01 = kpair(a.x, ca, hi2, lo2), k23 = kpair(a.y, ca, hi2, lo2);
  const uint32_t k45 = kpair(a.z, cb, hi2, lo2), k67 = kpair(a.w, cb, hi2, lo2);
  // magnitudes: element b of the low level-3 group -> low nibble of byte b,
  // element 4+b -> high nibble of byte b
  const uint32_t lo = __builtin_amdgcn_perm(k23, k01, 0x06040200u);
  const uint32_t hi = __builtin_amdgcn_perm(k67, k45, 0x06040200u);
  const uint32_t mag = lo | (hi << 4);
  // signs: the high byte of each bf16 carries its sign in bit 7
  const uint32_t sl = __builtin_amdgcn_perm(w.y, w.x, 0x07050301u);  // elements 0..3
  const uint32_t sh = __builtin_amdgcn_perm(w.w, w.z, 0x07050301u);  // elements 4..7
  const uint32_t sgn = ((sl >> 4) & 0x08080808u) | (sh & 0x80808080u);
  // a zero element keeps +0: sign only where the magnitude nibble is nonzero
  const uint32_t nz = (mag + 0x77777777u) & 0x88888888u;
  return mag | (sgn & nz);
}

// Nonzero bytes of a 32-bit word -> bits 0..3.
__device__ __forceinline__ uint32_t nonzero_bytes(uint32_t w) {
  const uint32_t hi = (((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w) & 0x80808080u;
  return ((hi >> 7) | (hi >> 14) | (hi >> 21) | (hi >> 28)) & 0xFu;
}

// One 16-element item (two level-2 groups, words v0 and v1, element 2i in
// the low half of word i; protected channels already cleared to +0, so they
// do not enter the maxima): item j of its row, it = its index over all rows
// (code words 2it, 2it+1; the unit's meta word it/4, written by the quad's
// first lane). Steps 1-5 of the rule.
__device__ __forceinline__ void quantize_item(uint4 v0, uint4 v1, uint32_t j, uint32_t it,
                                              uint32_t* __restrict__ codes32,
                                              uint32_t* __restrict__ meta) {
  const uint32_t q = j & 3u;  // item within the unit (groups 2q, 2q+1)

  // step 1: level-3 / level-2 maxima of |x| as bf16 bit patterns (sign bits
  // dropped; monotone in |x|), then the unit maximum over the quad of lanes
  const uint4 a0 = make_uint4(v0.x & 0x7FFF7FFFu, v0.y & 0x7FFF7FFFu, v0.z & 0x7FFF7FFFu,
                              v0.w & 0x7FFF7FFFu);
  const uint4 a1 = make_uint4(v1.x & 0x7FFF7FFFu, v1.y & 0x7FFF7FFFu, v1.z & 0x7FFF7FFFu,
                              v1.w & 0x7FFF7FFFu);
  const QuadMax q0 = quad_max(a0), q1 = quad_max(a1);
  const uint32_t am = max(max(q0.a, q0.b), max(q1.a, q1.b));
  const float amax = __uint_as_float(max4_u32(am) << 16);

  // step 2: level-1 code (shared by the quad)
  const uint32_t c = level1_code(amax);
  const float s = e6m2_f32(c);
  const uint32_t thr2 = __float_as_uint(3.5f * s) >> 16;
  const uint32_t thr175 = __float_as_uint(1.75f * s) >> 16;
  const uint32_t hi2 = kinv_hi2(c & 3u), lo2 = kinv_lo2(c & 3u);

  uint32_t e2a, e3a0, e3b0, e2b, e3a1, e3b1;
  const uint32_t cw0 = encode_group(v0, a0, q0, c >> 2, hi2, lo2, thr2, thr175, e2a, e3a0, e3b0);
  const uint32_t cw1 = encode_group(v1, a1, q1, c >> 2, hi2, lo2, thr2, thr175, e2b, e3a1, e3b1);

  reinterpret_cast<uint2*>(codes32)[it] = make_uint2(cw0, cw1);
  const uint32_t g0 = 2 * q, g1 = 2 * q + 1;
  const uint32_t mb = (e2a << (8 + g0)) | (e2b << (8 + g1)) | (e3a0 << (16 + 2 * g0)) |
                      (e3b0 << (17 + 2 * g0)) | (e3a1 << (16 + 2 * g1)) |
                      (e3b1 << (17 + 2 * g1));
  const uint32_t mw = or4_u32(mb) | c;
  if (q == 0u) meta[it >> 2] = mw;
}

// Kept values of one item of row `row`, one protected channel at a time:
// `info` = the item's 16 mask bits (high half) and the rank of its first
// masked channel among all masked channels (low half); the bf16 value of
// channel e goes to kept[row][rank of e].
__device__ __forceinline__ void keep_item_values(uint4 w0, uint4 w1, uint32_t info,
                                                 uint32_t row, uint16_t* __restrict__ kept,
                                                 int n_mask) {
  const uint32_t m16 = info >> 16;
  if (m16) {  // only lanes whose channels include masked ones
    const uint32_t ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    uint32_t mm = m16;
    while (mm) {
      const uint32_t e = __ffs(mm) - 1;
      const uint32_t rank = (info & 0xFFFFu) + __popc(m16 & ((1u << e) - 1u));
      if (rank < (uint32_t)n_mask)
        kept[(int64_t)row * n_mask + rank] = (uint16_t)(ww[e >> 1] >> (16 * (e & 1)));
      mm &= mm - 1;
    }
  }
}

}  // namespace hif4
