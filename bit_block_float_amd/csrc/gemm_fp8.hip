// gemm_fp8.hip -- Y = X W^T on E4M3 codes with a scale per block of 128 along
// K, on gfx950's scaled matrix cores.
//
// Y[i][j] = sum_b sx[i][b] sw[j][b] sum_{t in block b} cx[i][t] cw[j][t].
// sx is a power of two (E8M0), and so is sw where the library quantized it.
//
// Which matrix instruction, by the type of Y (beyond 16 rows; up to there the bf16
// forms cost next to nothing, see gemm_fp8_skinny_kernel):
//  - bf16: v_mfma_scale_f32_32x32x64_f8f6f4 on the codes as they are, both E8M0
//    bytes applied by the instruction. Measured on gfx950 (and the same for the
//    unscaled fp8 forms): within each run of 8 consecutive K values a product
//    is cut to a multiple of 2^-13 of the largest one's power of two before the
//    8 are added; the runs and the accumulator add in full fp32. The loss is at
//    most 7 * 2^-13 of each run's largest product, on random signs some 1e-5 of
//    |Y|: far below the 2^-8 rounding of a bf16 result, and half the time. (Where a
//    run's large products cancel, its small ones are lost: hif4.h says so, and that
//    a float32 Y has them.)
//  - fp32: the codes are widened to bf16 (v_cvt_scalef32_pk_bf16_fp8, with the
//    power-of-two scale applied: exact for scale bytes 3 to 246; below, bf16 has no
//    bits under 2^-133 and rounds, above, its range ends) and multiplied by the bf16
//    forms, whose products and sums are full fp32, subnormal operands included: a
//    float32 result is asked for where the last bits count.
// A weight whose scales are float32 (one per 128 x 128) keeps sx in the
// operands and adds each block's partial sum times sw with one FMA per output.
//
// The MFMA's first operand is W, so a lane of the result holds one row of Y
// (its column index) and runs of 4 consecutive columns.
#include <algorithm>
#include <type_traits>

#include "fp8_dev.h"

namespace hif4 {

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(8))) __bf16 gbf16x8_t;
typedef __attribute__((ext_vector_type(4))) uint32_t bf16x8_words_t;
typedef __attribute__((ext_vector_type(4))) uint32_t gu32x4_t;
typedef __attribute__((ext_vector_type(2))) uint32_t gu32x2_t;
typedef __attribute__((ext_vector_type(16))) float gf32x16_t;
typedef __attribute__((ext_vector_type(4))) float gf32x4_t;
typedef __attribute__((address_space(3))) void glds_void_t;

constexpr int kFmtE4M3 = 0;     // cbsz / blgp of the f8f6f4 forms
constexpr int kUnitScale = 127; // E8M0 byte of 1.0
constexpr int kRsrc3 = 0x00020000;

__device__ __forceinline__ i32x8_t join(gu32x4_t a, gu32x4_t b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

__device__ __forceinline__ gf32x16_t mfma32(i32x8_t a, i32x8_t b, gf32x16_t c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, kFmtE4M3, kFmtE4M3, 0, sa, 0, sb);
}

// This wave's loads but the newest n have landed, its LDS reads are done.
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n == 0 || n == 5 || n == 10, "one asm a count");
  if constexpr (n == 0) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  if constexpr (n == 5) asm volatile("s_waitcnt vmcnt(5) lgkmcnt(0)" ::: "memory");
  if constexpr (n == 10) asm volatile("s_waitcnt vmcnt(10) lgkmcnt(0)" ::: "memory");
}

// Direct-to-LDS loads of 16 (4) bytes a lane, to `dst` + 16 (4) * lane.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (glds_void_t*)dst, 16, voff, off, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (glds_void_t*)dst, 4, voff, off, 0, 0);
}

// 8 codes (two words) as bf16 times the power of two `s`.
__device__ __forceinline__ gbf16x8_t widen(uint32_t lo, uint32_t hi, float s) {
  const bf16x8_words_t w = {
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true))};
  return __builtin_bit_cast(gbf16x8_t, w);
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
__device__ __forceinline__ void store_tile(const gf32x16_t (&acc)[kTN][kTM], char* stage, void* Y,
                                           int64_t row0, int64_t col0, int64_t M, int64_t N,
                                           int lane) {
  constexpr int kE = kBf16 ? 2 : 4, kPer = 16 / kE;          // elements a 16-byte piece
  constexpr int kPitch = kTN * 32 * kE + 16;                 // rows start 4 banks apart
  constexpr int kLanes = kTN * 32 * kE / 16;                 // pieces a row
  constexpr int kRows = 64 / kLanes;                         // rows an instruction
  const bool vec = (N & (kPer - 1)) == 0 && ((uintptr_t)Y & 15) == 0;
  const bool whole = vec && row0 + 32 * kTM <= M && col0 + 32 * kTN <= N;  // uniform
  char* const put = stage + (lane & 31) * kPitch + (lane >> 5) * 4 * kE;
  const char* const get = stage + (lane / kLanes) * kPitch + (lane % kLanes) * 16;
  const int64_t col = col0 + (lane % kLanes) * kPer;
#pragma unroll
  for (int j = 0; j < kTM; ++j) {
#pragma unroll
    for (int i = 0; i < kTN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const gf32x16_t& a = acc[i][j];
        char* dst = put + (i * 32 + 8 * g) * kE;
        if constexpr (kBf16)
          *reinterpret_cast<gu32x2_t*>(dst) =
              gu32x2_t{f32x2_to_bf16x2(a[4 * g], a[4 * g + 1]),
                       f32x2_to_bf16x2(a[4 * g + 2], a[4 * g + 3])};
        else
          *reinterpret_cast<gf32x4_t*>(dst) =
              gf32x4_t{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
      }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < 32 / kRows; ++p) {
      const gu32x4_t v = *reinterpret_cast<const gu32x4_t*>(get + p * kRows * kPitch);
      const int64_t row = row0 + j * 32 + p * kRows + lane / kLanes;
      char* dst = reinterpret_cast<char*>(Y) + (row * N + col) * kE;
      if (whole || (vec && row < M && col + kPer <= N)) {
        __builtin_nontemporal_store(v, reinterpret_cast<gu32x4_t*>(dst));
      } else if (row < M) {
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
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
}

// Tile (row, column) of workgroup t: consecutive workgroup ids go to different
// XCDs; each XCD gets a contiguous run of tiles, walked column by column in
// groups of 4 tile rows (57600 x 13824 x 5120: 3.03 ms; groups of 8 3.05, of 16 3.17).
__device__ __forceinline__ void tile_of(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, int64_t& tm,
                                        int64_t& tn) {
  const uint32_t per_xcd = tiles_m * tiles_n / 8;
  if (t < per_xcd * 8) t = (t & 7) * per_xcd + (t >> 3);
  const uint32_t group = 4, per_group = group * tiles_n;
  const uint32_t gi = t / per_group, first = gi * group, in = t - gi * per_group;
  const uint32_t gsize = min(tiles_m - first, group);
  tm = __builtin_amdgcn_readfirstlane(first + in % gsize);
  tn = __builtin_amdgcn_readfirstlane(in / gsize);
}

// A product, cut into tiles_m x tiles_n tiles of Y.
struct GemmArgs {
  const uint8_t *x, *xs;
  int64_t ldxs;
  const uint8_t* w;
  const void* ws;  // E8M0 bytes, or float32
  int64_t ldws;
  int w_shift;
  int64_t m, n;
  int k;
  void* y;
  uint32_t tiles_m, tiles_n;
};

// Tile kernel, for products too small for the one below, and for float32 weight
// scales (57600 x 13824 x 5120: bf16 Y 4.2 ms, 1.94 PFLOP/s, with one FMA an output
// and block beside the products; fp32 Y 7.5 ms). BM x BN of Y a workgroup, kWM x
// kWN waves. A stage is one block of 128 along K: rows of 128 bytes = 8 chunks of 16, chunk c of row r in slot
// c ^ ((r >> 1) & 7), so that the fragment reads of 16 consecutive rows land in
// distinct bank groups. kStages of them are in LDS, brought by direct-to-LDS
// buffer loads, 8 rows an instruction, with the swizzle applied to the global
// address; rows past M or N fail the buffer's range check and read as zero. With
// each stage a wave brings one group of 64 scale words (the 4 bytes that hold the
// block's). Loads past the last block repeat it, into stages that no one reads.
//
// Part `split`: blocks [split per_split, (split + 1) per_split) of K only, the sums
// to that plane of Y as float32 (few tiles and a long K: the parts are added by
// gemm_fp8_reduce_kernel in order).
template <int BM, int BN, int kStages>
constexpr int kTileLds = kStages * (BM + BN) * (128 + 4) + 256;  // stages, a sink for idle scale loads
template <int BM, int BN, int kWM, int kWN, int kStages, bool kF32Scale, bool kFp8, bool kBf16>
__device__ __forceinline__ void gemm_fp8_tile(const GemmArgs& a, uint32_t tile, int split,
                                              int per_split, char* const lds) {
  const uint8_t* __restrict__ const X = a.x;
  const uint8_t* __restrict__ const XS = a.xs;
  const uint8_t* __restrict__ const W = a.w;
  const void* __restrict__ const WS = a.ws;
  const int64_t ldxs = a.ldxs, ldws = a.ldws, M = a.m, N = a.n;
  const int w_shift = a.w_shift, K = a.k;
  constexpr int kWaves = kWM * kWN;
  constexpr int kTM = BM / kWM / 32, kTN = BN / kWN / 32;  // 32 x 32 blocks of a wave
  constexpr int kCodes = (BM + BN) * 128, kStage = kCodes + (BM + BN) * 4;
  constexpr int kGroups = (kF32Scale ? BM : BM + BN) / 64;  // of 64 scale words
  static_assert(kGroups <= kWaves, "one group a wave");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  int64_t m0, n0;
  tile_of(tile, a.tiles_m, a.tiles_n, m0, n0);
  m0 *= BM;
  n0 *= BN;
  const int kb0 = split * per_split, kb1 = min(kb0 + per_split, K / 128);

  const int mrows = (int)min((int64_t)BM, M - m0), nrows = (int)min((int64_t)BN, N - n0);
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc((void*)(X + m0 * K), (short)0, mrows * K, kRsrc3);
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc((void*)(W + n0 * K), (short)0, nrows * K, kRsrc3);
  // this wave's scale words: X rows (groups 0 ..), then W rows; waves without a
  // group read X's first row into the sink
  const bool has = wave < kGroups, of_x = wave < BM / 64 || !has;
  const uint32_t srow = has ? (of_x ? wave * 64 + lane : ((wave - BM / 64) * 64 + lane) >> w_shift) : 0u;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(of_x ? XS + m0 * ldxs : (const uint8_t*)WS + (n0 >> w_shift) * ldws), (short)0,
      (int)(of_x ? mrows * ldxs : (((nrows - 1) >> w_shift) + 1) * ldws), kRsrc3);
  const uint32_t soff = srow * (uint32_t)(of_x ? ldxs : ldws);

  constexpr int kLoads = (BM + BN) / 8 / kWaves;  // of codes, per wave and stage
  constexpr int kXLoads = BM / 8 / kWaves;
  static_assert((BM + BN) % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole loads a wave");
  uint32_t voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = (i < kXLoads ? wave * kXLoads + i : wave * (kLoads - kXLoads) + i - kXLoads) * 8 +
                    (lane >> 3);
    voff[i] = (uint32_t)row * (uint32_t)K + (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }
  auto load_stage = [&](int kb, int slot) {
    char* base = lds + slot * kStage;
    const int blk = min(kb, kb1 - 1);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < kXLoads)
        load_lds16(rx, base + (wave * kXLoads + i) * 1024, voff[i], blk * 128);
      else
        load_lds16(rw, base + BM * 128 + (wave * (kLoads - kXLoads) + i - kXLoads) * 1024, voff[i],
                   blk * 128);
    }
    load_lds4(rs, has ? base + kCodes + wave * 256 : lds + kStages * kStage, soff, (blk >> 2) * 4);
  };

  gf32x16_t acc[kTN][kTM];
#pragma unroll
  for (int i = 0; i < kTN; ++i)
#pragma unroll
    for (int j = 0; j < kTM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int frow = lane & 31, fhalf = lane >> 5, fsw = (frow >> 1) & 7;
  const int xrow = wm * (BM / kWM) + frow, wrow = wn * (BN / kWN) + frow;
  // kF32Scale: the wave's one block row (the last one where all its columns are past N)
  const float* wsf = reinterpret_cast<const float*>(WS) +
                     (min(n0 + wn * (BN / kWN), N - 1) >> 7) * ldws;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load_stage(kb0 + s, s);
  int slot = 0;
  for (int kb = kb0; kb < kb1; ++kb) {
    // stage kb has landed for this wave (the loads of the kStages - 2 after it may
    // be in flight); after the barrier for all, and every wave has read the stage
    // that is loaded next
    wait_loads<(kStages - 2) * (kLoads + 1)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_stage(kb + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
    const char* const stage = lds + slot * kStage;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    uint32_t sxw[kTM], sww[kTN];
#pragma unroll
    for (int j = 0; j < kTM; ++j)
      sxw[j] = *reinterpret_cast<const uint32_t*>(stage + kCodes + (xrow + j * 32) * 4);
    if constexpr (!kF32Scale) {
#pragma unroll
      for (int i = 0; i < kTN; ++i)
        sww[i] = *reinterpret_cast<const uint32_t*>(stage + kCodes + (BM + wrow + i * 32) * 4);
    }
    const int sh = 8 * (kb & 3);
    const char* xs = stage + xrow * 128;
    const char* ws = stage + (BM + wrow) * 128;
    float wscale = 0.0f;
    if constexpr (kF32Scale) wscale = wsf[kb];
    auto chunk = [&](const char* row, int c) {
      return *reinterpret_cast<const gu32x4_t*>(row + ((c ^ fsw) * 16));
    };
    if constexpr (kFp8) {
      // half s of the block: lanes 0..31 chunks 4s, 4s + 1, lanes 32..63 the next two
      auto frag = [&](const char* row, int s) {
        return join(chunk(row, 4 * s + 2 * fhalf), chunk(row, 4 * s + 2 * fhalf + 1));
      };
      if constexpr (!kF32Scale) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          i32x8_t fx[kTM];
#pragma unroll
          for (int j = 0; j < kTM; ++j) fx[j] = frag(xs + j * 4096, s);
#pragma unroll
          for (int i = 0; i < kTN; ++i) {
            const i32x8_t fw = frag(ws + i * 4096, s);
#pragma unroll
            for (int j = 0; j < kTM; ++j)
              acc[i][j] = mfma32(fw, fx[j], acc[i][j], (int)(sww[i] >> sh), (int)(sxw[j] >> sh));
          }
        }
      } else {
        i32x8_t fx[2][kTM];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < kTM; ++j) fx[s][j] = frag(xs + j * 4096, s);
#pragma unroll
        for (int i = 0; i < kTN; ++i) {
          const i32x8_t w0 = frag(ws + i * 4096, 0), w1 = frag(ws + i * 4096, 1);
#pragma unroll
          for (int j = 0; j < kTM; ++j) {
            gf32x16_t p = {0.0f};
            p = mfma32(w0, fx[0][j], p, kUnitScale, (int)(sxw[j] >> sh));
            p = mfma32(w1, fx[1][j], p, kUnitScale, (int)(sxw[j] >> sh));
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(p[r], wscale, acc[i][j][r]);
          }
        }
      }
    } else {
      // chunk pair q: lanes 0..31 chunk 2q, lanes 32..63 chunk 2q + 1, 16 codes
      // each = the operands of two MFMAs
      float sxf[kTM], swf[kTN];
#pragma unroll
      for (int j = 0; j < kTM; ++j) sxf[j] = e8m0_f32((sxw[j] >> sh) & 255u);
#pragma unroll
      for (int i = 0; i < kTN; ++i) swf[i] = kF32Scale ? 1.0f : e8m0_f32((sww[i] >> sh) & 255u);
      if constexpr (!kF32Scale) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          gbf16x8_t fx[2][kTM];
#pragma unroll
          for (int j = 0; j < kTM; ++j) {
            const gu32x4_t v = chunk(xs + j * 4096, 2 * q + fhalf);
            fx[0][j] = widen(v.x, v.y, sxf[j]);
            fx[1][j] = widen(v.z, v.w, sxf[j]);
          }
#pragma unroll
          for (int i = 0; i < kTN; ++i) {
            const gu32x4_t v = chunk(ws + i * 4096, 2 * q + fhalf);
            const gbf16x8_t w0 = widen(v.x, v.y, swf[i]), w1 = widen(v.z, v.w, swf[i]);
#pragma unroll
            for (int j = 0; j < kTM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w0, fx[0][j], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < kTM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w1, fx[1][j], acc[i][j], 0, 0, 0);
          }
        }
      } else {
        // one row block at a time: the partial sums of all would not fit beside
        // the accumulators
#pragma unroll
        for (int j = 0; j < kTM; ++j) {
          gf32x16_t p[kTN];
#pragma unroll
          for (int i = 0; i < kTN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) p[i][r] = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const gu32x4_t v = chunk(xs + j * 4096, 2 * q + fhalf);
            const gbf16x8_t x0 = widen(v.x, v.y, sxf[j]), x1 = widen(v.z, v.w, sxf[j]);
#pragma unroll
            for (int i = 0; i < kTN; ++i) {
              const gu32x4_t u = chunk(ws + i * 4096, 2 * q + fhalf);
              p[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(u.x, u.y, 1.0f), x0, p[i], 0, 0, 0);
              p[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen(u.z, u.w, 1.0f), x1, p[i], 0, 0, 0);
            }
          }
#pragma unroll
          for (int i = 0; i < kTN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(p[i][r], wscale, acc[i][j][r]);
        }
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  static_assert(kWaves * kStageBytes<kBf16, kTN> <= kTileLds<BM, BN, kStages>, "epilogue stage");
  char* const y = reinterpret_cast<char*>(a.y) + split * M * N * (kBf16 ? 2 : 4);
  store_tile<kBf16, kTN, kTM>(acc, lds + wave * kStageBytes<kBf16, kTN>, y, m0 + wm * (BM / kWM),
                              n0 + wn * (BN / kWN), M, N, lane);
}

template <int BM, int BN, int kWM, int kWN, int kStages, bool kF32Scale, bool kFp8, bool kBf16>
__global__ __launch_bounds__(kWM* kWN * 64) void gemm_fp8_tile_kernel(GemmArgs a, int per_split) {
  __shared__ __attribute__((aligned(1024))) char lds[kTileLds<BM, BN, kStages>];
  gemm_fp8_tile<BM, BN, kWM, kWN, kStages, kF32Scale, kFp8, kBf16>(a, blockIdx.x, (int)blockIdx.y,
                                                                  per_split, lds);
}

// Two products in one launch, the first with `first` tiles: few tiles leave CUs idle
// that the second's can have.
template <int BM, int BN, int kWM, int kWN, int kStages, bool kBf16A, bool kBf16B>
__global__ __launch_bounds__(kWM* kWN * 64) void gemm_fp8_tile_pair_kernel(GemmArgs a, GemmArgs b,
                                                                           uint32_t first) {
  __shared__ __attribute__((aligned(1024))) char lds[kTileLds<BM, BN, kStages>];
  if (blockIdx.x < first)
    gemm_fp8_tile<BM, BN, kWM, kWN, kStages, false, kBf16A, kBf16A>(a, blockIdx.x, 0, a.k / 128, lds);
  else
    gemm_fp8_tile<BM, BN, kWM, kWN, kStages, false, kBf16B, kBf16B>(b, blockIdx.x - first, 0,
                                                                    b.k / 128, lds);
}

// Y = sum of `splits` float32 planes, in order; 4 elements a thread.
template <bool kBf16>
__global__ __launch_bounds__(256) void gemm_fp8_reduce_kernel(const float* __restrict__ parts,
                                                              int splits, int64_t total,
                                                              void* __restrict__ Y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  if (i + 4 <= total && (total & 3) == 0) {
    gf32x4_t s = *reinterpret_cast<const gf32x4_t*>(parts + i);
    for (int p = 1; p < splits; ++p) s += *reinterpret_cast<const gf32x4_t*>(parts + p * total + i);
    if constexpr (kBf16)
      *reinterpret_cast<gu32x2_t*>(reinterpret_cast<uint16_t*>(Y) + i) =
          gu32x2_t{f32x2_to_bf16x2(s[0], s[1]), f32x2_to_bf16x2(s[2], s[3])};
    else
      *reinterpret_cast<gf32x4_t*>(reinterpret_cast<float*>(Y) + i) = s;
  } else {
    for (int64_t e = i; e < min(i + 4, total); ++e) {
      float s = parts[e];
      for (int p = 1; p < splits; ++p) s += parts[p * total + e];
      if constexpr (kBf16) reinterpret_cast<uint16_t*>(Y)[e] = (uint16_t)f32_to_bf16(s);
      else reinterpret_cast<float*>(Y)[e] = s;
    }
  }
}

// Large products with E8M0 scales on both sides. 256 x 256 of Y a workgroup, 4
// waves of 128 x 128 (256 fp32 accumulators a lane), one workgroup a CU: against
// 8 waves of 128 x 64 a third less is read from LDS per product, and LDS would
// be busy as long as the matrix cores.
//
// Bound: the matrix cores at the clock that the chip's power allows. Measured on
// 57600 x 13824 x 5120, bf16 Y: 2.95 to 3.21 ms (2.54 to 2.76 PFLOP/s), the matrix
// cores busy 73% of the cycles; without any load, LDS read or store it would take
// 2.1 ms. fp32 Y (bf16 instructions): 5.74 ms, 1.42 PFLOP/s. Workgroups that stay
// and run on from tile to tile, with the next tile's first blocks loaded ahead,
// were 1% to 4% slower.
//
// A stage is one block (128 K values): rows of 128 bytes, whole cache lines,
// chunk c of 16 bytes in slot c ^ ((row >> 1) & 7) (the reads of 16 consecutive
// rows land in distinct bank groups). Two stages are in LDS, each multiplied in
// two halves of 64 K values: while half 0 of block kb multiplies from registers,
// half 1 is read into the other register set; then one barrier, after which no
// wave needs the stage, and block kb + 2 goes out into it by direct-to-LDS loads
// while half 1 multiplies and half 0 of block kb + 1 is read. Blocks past the end
// load the last one again, into a stage that no one reads.
constexpr int kBigSlot = 2 * 256 * 128;
constexpr int kBigScaleRing = 2 * 256 * 4;
constexpr int kBigLds = 2 * kBigSlot + 2 * kBigScaleRing + 1024;  // + a sink for idle scale loads

template <bool kBf16>
__device__ __forceinline__ void gemm_fp8_big(const GemmArgs& a, uint32_t tile, char* const lds) {
  const uint8_t* __restrict__ const X = a.x;
  const uint8_t* __restrict__ const XS = a.xs;
  const uint8_t* __restrict__ const W = a.w;
  const uint8_t* __restrict__ const WS = (const uint8_t*)a.ws;
  const int64_t ldxs = a.ldxs, ldws = a.ldws, M = a.m, N = a.n;
  const int w_shift = a.w_shift, K = a.k;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  int64_t m0, n0;
  tile_of(tile, a.tiles_m, a.tiles_n, m0, n0);
  m0 *= 256;
  n0 *= 256;

  const int mrows = (int)min((int64_t)256, M - m0), nrows = (int)min((int64_t)256, N - n0);
  const __amdgpu_buffer_rsrc_t rx =
      __builtin_amdgcn_make_buffer_rsrc((void*)(X + m0 * K), (short)0, mrows * K, kRsrc3);
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc((void*)(W + n0 * K), (short)0, nrows * K, kRsrc3);
  const int xs_bytes = (int)(mrows * ldxs), ws_bytes = (int)((((nrows - 1) >> w_shift) + 1) * ldws);

  // loads: instruction i of a wave brings rows 64 wave + 8 (i & 7) .. + 7 of X (i < 8) or W
  uint32_t voff[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = wave * 64 + i * 8 + (lane >> 3);
    voff[i] = (uint32_t)row * (uint32_t)K + (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }
  const int KB = K / 128;
  auto load_part = [&](int kb, int i) {
    char* dst = lds + (kb & 1) * kBigSlot + (i >> 3) * 32768 + wave * 8192 + (i & 7) * 1024;
    const int off = min(kb, KB - 1) * 128;
    if (i < 8)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (glds_void_t*)dst, 16, voff[i & 7], off, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (glds_void_t*)dst, 16, voff[i & 7], off, 0, 0);
  };
  // Scale words of blocks 4g .. 4g + 3: a wave brings 64 rows of X's in block 4g - 4
  // and of W's in block 4g - 3. (One load a block, whose target is chosen without
  // a branch: a branch in the loop would let the compiler move products across
  // the step's barrier.)
  const uint32_t xs_off = (uint32_t)(wave * 64 + lane) * (uint32_t)ldxs;
  const uint32_t ws_off = (uint32_t)((wave * 64 + lane) >> w_shift) * (uint32_t)ldws;
  const int last_group = (KB - 1) >> 2;
  char* const scale_ring = lds + 2 * kBigSlot;
  auto load_scale = [&](int kb) {
    const int g = min((kb >> 2) + 1, last_group), part = kb & 3;
    char* dst = part < 2 ? scale_ring + (((kb >> 2) + 1) & 1) * kBigScaleRing + part * 1024
                         : scale_ring + 2 * kBigScaleRing;
    const bool is_w = (part & 1) != 0;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(is_w ? WS + (n0 >> w_shift) * ldws : XS + m0 * ldxs), (short)0,
        is_w ? ws_bytes : xs_bytes, kRsrc3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (glds_void_t*)(dst + wave * 256), 4,
                                             is_w ? ws_off : xs_off, 4 * g, 0, 0);
  };

  const int frow = lane & 31, fhalf = lane >> 5, fsw = (frow >> 1) & 7;
  const char* const xbase = lds + (wm * 128 + frow) * 128;
  const char* const wbase = lds + 32768 + (wn * 128 + frow) * 128;
  // fragments of half a block: blocks of 32 rows 0..3 of X, 4..7 of W, two chunks each
  struct Frags {
    gu32x4_t v[8][2];
  };
  int slot[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 2; ++e) slot[s][e] = ((4 * s + 2 * fhalf + e) ^ fsw) * 16;
  auto read_part = [&](Frags& f, int kb, int s, int p) {  // p = 0..15
    const char* base = ((p >> 1) < 4 ? xbase : wbase) + (kb & 1) * kBigSlot + ((p >> 1) & 3) * 4096;
    f.v[p >> 1][p & 1] = *reinterpret_cast<const gu32x4_t*>(base + slot[s][p & 1]);
  };
  uint32_t sw[8];  // this block's scale bytes (low byte): X blocks, W blocks
  uint32_t snext[8];
  auto read_scale = [&](int kb, int b) {  // the word that holds block kb's byte
    const char* base = scale_ring + ((kb >> 2) & 1) * kBigScaleRing + (b < 4 ? 0 : 1024);
    snext[b] = *reinterpret_cast<const uint32_t*>(
        base + ((b < 4 ? wm : wn) * 128 + (b & 3) * 32 + frow) * 4);
  };

  gf32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  load_scale(-4);
  load_scale(-3);
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) load_part(kb, i);
  asm volatile("s_waitcnt vmcnt(16)" ::: "memory");  // scales and block 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags f0, f1;
#pragma unroll
  for (int p = 0; p < 16; ++p) read_part(f0, 0, 0, p);
#pragma unroll
  for (int b = 0; b < 8; ++b) read_scale(0, b);

  // one half (s of block kb): the products of `cur`, the other half's fragments
  // into `nxt`, and in half 1 the loads of block kb + 2
  auto half = [&](const Frags& cur, Frags& nxt, int kb, auto s, const uint32_t (&sc)[8]) {
    constexpr int kS = decltype(s)::value;
    auto reads = [&](int p) { read_part(nxt, kb + kS, 1 - kS, p); };
    if constexpr (kBf16) {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        // Half 0 reads first: the barrier waits for the last read. Half 1 sends one
        // load a product: bursts of two cost 6% (a wave whose loads back up in the
        // memory pipeline issues no products either).
        if (kS == 0 ? c < 8 : c >= 2 && c < 10) {
          reads(2 * (c - 2 * kS));
          reads(2 * (c - 2 * kS) + 1);
        }
        if constexpr (kS == 1) load_part(kb + 2, c);
        const int i = c >> 2, j = c & 3;
        acc[i][j] = mfma32(join(cur.v[4 + i][0], cur.v[4 + i][1]), join(cur.v[j][0], cur.v[j][1]),
                           acc[i][j], (int)sc[4 + i], (int)sc[j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      float sf[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) sf[b] = e8m0_f32(sc[b] & 255u);
      gbf16x8_t d[2][8];  // widened operands of 16 K values a lane pair, two sets in turn
#pragma unroll
      for (int b = 0; b < 8; ++b) d[0][b] = widen(cur.v[b][0].x, cur.v[b][0].y, sf[b]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (c < 4) reads(4 * q + c);
          if constexpr (kS == 1) {
            if (c >= 4 && c < 12 && (c & 1) == 0) load_part(kb + 2, 4 * q + ((c - 4) >> 1));
          }
          if (q < 3 && (c & 1)) {
            const gu32x4_t v = cur.v[c >> 1][(q + 1) >> 1];
            d[(q + 1) & 1][c >> 1] = ((q + 1) & 1) ? widen(v.z, v.w, sf[c >> 1]) : widen(v.x, v.y, sf[c >> 1]);
          }
          const int i = c >> 2, j = c & 3;
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d[q & 1][4 + i], d[q & 1][j],
                                                              acc[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  using H0 = std::integral_constant<int, 0>;
  using H1 = std::integral_constant<int, 1>;
  for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
    for (int b = 0; b < 8; ++b) sw[b] = snext[b] >> (8 * (kb & 3));
    half(f0, f1, kb, H0{}, sw);
    // block kb is in registers everywhere, block kb + 1 has landed
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_scale(kb);
#pragma unroll
    for (int b = 0; b < 8; ++b) read_scale(kb + 1, b);
    half(f1, f0, kb, H1{}, sw);
  }
  // every load has landed and every wave has read what it will: the stages are free
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  static_assert(4 * kStageBytes<kBf16, 4> <= kBigLds, "epilogue stage");
  store_tile<kBf16, 4, 4>(acc, lds + wave * kStageBytes<kBf16, 4>, a.y, m0 + wm * 128, n0 + wn * 128,
                          M, N, lane);
}

template <bool kBf16>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_big_kernel(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[kBigLds];
  gemm_fp8_big<kBf16>(a, blockIdx.x, lds);
}

// Two products in one launch, `first` workgroups of the first: the CUs that the
// first one's last round of tiles leaves idle begin with the second. Measured on
// the two gradients of an 8192 x 5120 x 5120 layer (400 tiles of fp32 dW, 640 of
// bf16 dX), best of nine: two launches 353 + 188 us, one 487 us.
template <bool kBf16A, bool kBf16B>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_pair_kernel(GemmArgs a, GemmArgs b, uint32_t first) {
  __shared__ __attribute__((aligned(1024))) char lds[kBigLds];
  if (blockIdx.x < first) gemm_fp8_big<kBf16A>(a, blockIdx.x, lds);
  else gemm_fp8_big<kBf16B>(b, blockIdx.x - first, lds);
}

// Up to 16 rows: bound by reading W once. A workgroup owns `cols` <= 16 columns of
// Y; its waves take the K blocks in turn, W straight from memory into the MFMA's
// operand registers, and their sums meet in LDS in a fixed order. Rows past M or
// the workgroup's columns repeat the last one and are not stored.
//
// The codes are widened to bf16 without their scales (exact), so a block's sum is a
// full fp32 sum of exact products for either type of Y; then its two scales are
// applied as one exponent (a float scale's significand by the FMA that adds the
// block), so that only the result has to be in fp32's range. The fp8 instructions,
// which would cut products, gain little, W's bytes being what counts. With six
// weights in turn, they and this, us: float32 scales 1 x 13824 x 5120 14.4 and 14.9, 16
// x 13824 x 5120 24.5 and 24.6; E8M0 tiles 1 x 5120 x 13824 18.3 and 17.2, 16 x 13824 x
// 5120 25.0 and 24.9; E8M0 rows 25.8 and 26.9.
//
// What a CU can have in flight to memory sets the pace, so the columns are cut to
// give every CU the same share: cols is the least that leaves as many workgroups
// a CU as 16 would. Measured, one row: n = 5120, k = 13824, 320 workgroups of 16
// columns 17.9 us, 512 of 10 15.3 us; n = 13824, k = 5120, 864 of 16 14.5 us, 988
// of 14 13.6 us. (16 rows against tiles, n = k = 5120: 10.9 and 12.0 us; 24 rows
// the other way about, 14.3 and 12.0 us.)
constexpr int kSkinnyRows = 16;
constexpr int kSkinnyWaves = 16;
// kTiles: W's scales are one per 128 x 128, float32 or E8M0; else E8M0 bytes per row.
template <bool kTiles, bool kF32Scale, bool kBf16>
__global__ __launch_bounds__(kSkinnyWaves * 64) void gemm_fp8_skinny_kernel(
    const uint8_t* __restrict__ X, const uint8_t* __restrict__ XS, int64_t ldxs,
    const uint8_t* __restrict__ W, const void* __restrict__ WS, int64_t ldws, int M, int64_t N,
    int K, int cols, void* __restrict__ Y) {
  static_assert(kTiles || !kF32Scale, "float32 scales are per 128 x 128");
  __shared__ gf32x4_t part[kSkinnyWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * cols, n1 = min(n0 + cols, N);
  const int64_t wr = min(n0 + r16, n1 - 1);
  const int xr = min(r16, M - 1);
  // of each block lane group kq takes bytes 16 kq and 64 + 16 kq on, of both operands
  const uint8_t* wp = W + wr * K + kq * 16;
  const uint8_t* xp = X + (int64_t)xr * K + kq * 16;
  const uint8_t* wsb = (const uint8_t*)WS + wr * ldws;
  const uint8_t* xsb = XS + (int64_t)xr * ldxs;
  // kTiles: the columns lie in one block row, or two
  const int64_t ws0 = (n0 >> 7) * ldws, ws1 = ((n1 - 1) >> 7) * ldws;
  auto scale_of = [&](int64_t row, int k) {  // as f 2^q: 1 <= |f| < 2 (a power of two: f = 1)
    struct { float f; int q; } r;
    if constexpr (kF32Scale) {
      const float s = reinterpret_cast<const float*>(WS)[row + k];
      r.f = 2.0f * __builtin_amdgcn_frexp_mantf(s);
      r.q = __builtin_amdgcn_frexp_expf(s) - 1;
    } else {
      const uint32_t b =
          reinterpret_cast<const uint32_t*>((const uint8_t*)WS + row)[k >> 2] >> (8 * (k & 3)) & 255u;
      r.f = b == 255u ? __uint_as_float(0x7FC00000u) : 1.0f;
      r.q = (int)b - 127;
    }
    return r;
  };
  const int64_t border = ((n1 - 1) >> 7) << 7;  // first column of the second
  gf32x4_t acc = {0, 0, 0, 0};
  const int KB = K / 128;
  // kU blocks at a time, their loads all in flight before the first product (past
  // the end the last block again, not used)
  constexpr int kU = 4;
  for (int kb = wave; kb < KB; kb += kU * kSkinnyWaves) {
    gu32x4_t w[kU][2], x[kU][2];
    uint32_t sw[kU], sx[kU];
    decltype(scale_of(0, 0)) t0[kU], t1[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int k = min(kb + u * kSkinnyWaves, KB - 1);
      w[u][0] = *reinterpret_cast<const gu32x4_t*>(wp + (int64_t)k * 128);
      w[u][1] = *reinterpret_cast<const gu32x4_t*>(wp + (int64_t)k * 128 + 64);
      x[u][0] = *reinterpret_cast<const gu32x4_t*>(xp + (int64_t)k * 128);
      x[u][1] = *reinterpret_cast<const gu32x4_t*>(xp + (int64_t)k * 128 + 64);
      sx[u] = xsb[k];
      if constexpr (kTiles) {
        t0[u] = scale_of(ws0, k);
        t1[u] = scale_of(ws1, k);
      } else {
        sw[u] = wsb[k];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (kb + u * kSkinnyWaves >= KB) break;  // uniform
      // the block's sum of code products, then its two scales, result by result
      gf32x4_t p = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(w[u][h].x, w[u][h].y, 1.0f),
                                                    widen(x[u][h].x, x[u][h].y, 1.0f), p, 0, 0, 0);
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(w[u][h].z, w[u][h].w, 1.0f),
                                                    widen(x[u][h].z, x[u][h].w, 1.0f), p, 0, 0, 0);
      }
      if constexpr (kTiles) {
        const float nan = __uint_as_float(0x7FC00000u);
        const float f0 = sx[u] == 255u ? nan : t0[u].f, f1 = sx[u] == 255u ? nan : t1[u].f;
        const int e0 = (int)sx[u] - 127 + t0[u].q, e1 = (int)sx[u] - 127 + t1[u].q;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool first = n0 + kq * 4 + r < border;
          acc[r] = fmaf(__builtin_amdgcn_ldexpf(p[r], first ? e0 : e1), first ? f0 : f1, acc[r]);
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // the column's operand is in lane kq * 4 + r
          const uint32_t swj = (uint32_t)__shfl((int)sw[u], kq * 4 + r, 64);
          acc[r] += max(sx[u], swj) == 255u ? __uint_as_float(0x7FC00000u)
                                            : __builtin_amdgcn_ldexpf(p[r], (int)(sx[u] + swj) - 254);
        }
      }
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    gf32x4_t s = part[0][lane];
#pragma unroll
    for (int w = 1; w < kSkinnyWaves; ++w) s += part[w][lane];
    const bool vec = (N & 3) == 0 && (cols & 3) == 0 && ((uintptr_t)Y & 15) == 0;
    const int64_t col = n0 + kq * 4;
    if (r16 < M && col < n1)
      store4<kBf16>(Y, (int64_t)r16 * N + col, (int)col, (int)n1, vec, s[0], s[1], s[2], s[3]);
  }
}

// Which kernel, from the sizes alone. Measured at k = 5120, bf16 Y (the same order
// with fp32), in us:
//   m x n           64 x 64   128, 2 a CU   128, 1 a CU   256 x 256
//   512 x 5120         32          31            26           50
//   512 x 13824        69          40            52           51
//   1024 x 5120        53          38            50           51
//   2048 x 5120        98          68            76           53
//   1024 x 13824      133          77           104           59
// A round of 256 tiles of 256 x 256 costs 4/3 of one of 512 tiles of 128 x 128.
// Splitting K pays for its second kernel from some 16 blocks a part: 300 x 700 x
// 13824 30 us whole, 20 in 2 parts, 16 in 4, 19 in 9; 200 x 2048 x 2048 8.0 us
// whole, 9.5 in 2.
enum GemmKind { kSkinny, kSmall, kOneRound, kMiddle, kLarge };
struct GemmPlan {
  GemmKind kind;
  int splits, per_split;  // of K's blocks
};
constexpr int64_t kCus = 256;
static GemmPlan plan_gemm(int64_t m, int64_t n, int64_t k) {  // k a multiple of 128, above 0
  const int64_t kb = k / 128;
  const auto tiles = [&](int64_t t) { return ((m + t - 1) / t) * ((n + t - 1) / t); };
  // (a grid has fewer than 2^32 threads: 1024 for 16 columns, so 2^22 - 1 workgroups)
  if (m <= kSkinnyRows && n <= (int64_t(1) << 26) - 16) return {kSkinny, 1, (int)kb};
  const int64_t t128 = tiles(128);
  if (4 * ((tiles(256) + kCus - 1) / kCus) < 3 * ((t128 + 2 * kCus - 1) / (2 * kCus)))
    return {kLarge, 1, (int)kb};
  if (t128 > kCus) return {kMiddle, 1, (int)kb};
  if (t128 >= kCus / 2) return {kOneRound, 1, (int)kb};
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(2 * kCus / tiles(64), kb / 16));
  const int64_t per = (kb + splits - 1) / splits;
  return {kSmall, (int)((kb + per - 1) / per), (int)per};
}

static GemmArgs gemm_args(const Fp8Product& p, int64_t tile, void* y) {
  return GemmArgs{p.x, p.xs, p.ldxs, p.w, p.ws, p.ldws, p.w_block == 128 ? 7 : 0, p.m, p.n, (int)p.k,
                  y, (uint32_t)((p.m + tile - 1) / tile), (uint32_t)((p.n + tile - 1) / tile)};
}

// The tile kernels by kind: tile rows and columns, waves both ways, stages.
#define HIF4_SMALL 64, 64, 2, 2, 4
#define HIF4_ONE_ROUND 128, 128, 2, 4, 3
#define HIF4_MIDDLE 128, 128, 2, 2, 2
#define HIF4_LARGE_F32 256, 256, 2, 4, 2

template <int BM, int BN, int kWM, int kWN, int kStages, bool kF32Scale, bool kFp8, bool kBf16>
static void launch_tiles(const Fp8Product& p, const GemmPlan& plan, void* y, hipStream_t stream) {
  const GemmArgs a = gemm_args(p, BM, y);
  hipLaunchKernelGGL((gemm_fp8_tile_kernel<BM, BN, kWM, kWN, kStages, kF32Scale, kFp8, kBf16>),
                     dim3(a.tiles_m * a.tiles_n, plan.splits), dim3(kWM * kWN * 64), 0, stream, a,
                     plan.per_split);
}

template <bool kF32Scale, bool kBf16>
static hipError_t launch_gemm(const Fp8Product& p, void* workspace, hipStream_t stream) {
  const GemmPlan plan = plan_gemm(p.m, p.n, p.k);
  switch (plan.kind) {
    case kSkinny: {
      const int64_t per_cu = (p.n + 16 * kCus - 1) / (16 * kCus);
      const int cols = (int)((p.n + kCus * per_cu - 1) / (kCus * per_cu));  // 1 .. 16
      const auto launch = [&](auto tiles) {
        hipLaunchKernelGGL((gemm_fp8_skinny_kernel<decltype(tiles)::value, kF32Scale, kBf16>),
                           dim3((unsigned)((p.n + cols - 1) / cols)), dim3(kSkinnyWaves * 64), 0,
                           stream, p.x, p.xs, p.ldxs, p.w, p.ws, p.ldws, (int)p.m, p.n, (int)p.k,
                           cols, p.y);
      };
      if constexpr (!kF32Scale) {
        if (p.w_block == 1) {
          launch(std::false_type{});
          break;
        }
      }
      launch(std::true_type{});
      break;
    }
    case kLarge:
      if constexpr (kF32Scale) {
        launch_tiles<HIF4_LARGE_F32, true, kBf16, kBf16>(p, plan, p.y, stream);
      } else {
        const GemmArgs a = gemm_args(p, 256, p.y);
        hipLaunchKernelGGL(gemm_fp8_big_kernel<kBf16>, dim3(a.tiles_m * a.tiles_n), dim3(256), 0,
                           stream, a);
      }
      break;
    case kMiddle: launch_tiles<HIF4_MIDDLE, kF32Scale, kBf16, kBf16>(p, plan, p.y, stream); break;
    case kOneRound: launch_tiles<HIF4_ONE_ROUND, kF32Scale, kBf16, kBf16>(p, plan, p.y, stream); break;
    case kSmall:
      if (plan.splits == 1) {
        launch_tiles<HIF4_SMALL, kF32Scale, kBf16, kBf16>(p, plan, p.y, stream);
        break;
      }
      launch_tiles<HIF4_SMALL, kF32Scale, kBf16, false>(p, plan, workspace, stream);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(gemm_fp8_reduce_kernel<kBf16>, dim3((unsigned)((p.m * p.n + 1023) / 1024)),
                         dim3(256), 0, stream, (const float*)workspace, plan.splits, p.m * p.n, p.y);
      break;
  }
  return hipGetLastError();
}

// Two products with E8M0 scales in one launch. false: not launched (too many tiles).
template <bool kBf16A, bool kBf16B>
static bool launch_pair(const Fp8Product& a, const Fp8Product& b, GemmKind kind, hipStream_t stream) {
  const int64_t tile = kind == kLarge ? 256 : kind == kSmall ? 64 : 128;
  const GemmArgs ga = gemm_args(a, tile, a.y), gb = gemm_args(b, tile, b.y);
  const uint64_t first = (uint64_t)ga.tiles_m * ga.tiles_n;
  const uint64_t all = first + (uint64_t)gb.tiles_m * gb.tiles_n;
  if (all >= (1ull << 24)) return false;  // a grid has fewer than 2^32 threads
#define HIF4_PAIR(kernel, threads)                                                        \
  hipLaunchKernelGGL((kernel), dim3((unsigned)all), dim3(threads), 0, stream, ga, gb, (uint32_t)first)
  switch (kind) {
    case kLarge: HIF4_PAIR((gemm_fp8_pair_kernel<kBf16A, kBf16B>), 256); return true;
    case kOneRound:
    case kMiddle: HIF4_PAIR((gemm_fp8_tile_pair_kernel<HIF4_MIDDLE, kBf16A, kBf16B>), 256); return true;
    case kSmall: HIF4_PAIR((gemm_fp8_tile_pair_kernel<HIF4_SMALL, kBf16A, kBf16B>), 256); return true;
    default: return false;
  }
#undef HIF4_PAIR
}

}  // namespace hif4

using namespace hif4;

hipError_t hif4_launch_gemm_fp8(const Fp8Product& p, void* workspace, hipStream_t stream) {
  if (p.ws_f32)
    return p.y_bf16 ? launch_gemm<true, true>(p, workspace, stream)
                    : launch_gemm<true, false>(p, workspace, stream);
  return p.y_bf16 ? launch_gemm<false, true>(p, workspace, stream)
                  : launch_gemm<false, false>(p, workspace, stream);
}

// Two independent products, in one launch where both have E8M0 scales and take the
// same kernel whole (two that fill the CUs once with one tile each: the kernel that
// has two a CU). Measured on the two gradients of a layer, two launches and one, us:
//   1024 x 1024 x 1024         11.0    7.7
//   1001 x 1300 x 640 (fp32)   13.5   11.1
//   2048 x 2048 x 2048         32.5   30.1 (as two rounds of one a CU: 35.3)
//   2100 x 2200 x 2111         63.9   53.7 (as tiles of 256: 61.1)
//   8192 x 5120 x 5120          541    487
// but with tiles that suit only one of them: 200 x 2048 x 2048 13.6 and 15.6,
// 4096 x 2048 x 2048 61.7 and 79.8.
hipError_t hif4_launch_gemm_fp8_two(const Fp8Product& a, const Fp8Product& b, void* workspace,
                                    hipStream_t stream) {
  const GemmPlan pa = plan_gemm(a.m, a.n, a.k), pb = plan_gemm(b.m, b.n, b.k);
  if (!a.ws_f32 && !b.ws_f32 && pa.kind == pb.kind && pa.splits == 1 && pb.splits == 1) {
    const bool done = a.y_bf16 ? (b.y_bf16 ? launch_pair<true, true>(a, b, pa.kind, stream)
                                           : launch_pair<true, false>(a, b, pa.kind, stream))
                               : (b.y_bf16 ? launch_pair<false, true>(a, b, pa.kind, stream)
                                           : launch_pair<false, false>(a, b, pa.kind, stream));
    if (done) return hipGetLastError();
  }
  const hipError_t e = hif4_launch_gemm_fp8(a, workspace, stream);
  return e != hipSuccess ? e : hif4_launch_gemm_fp8(b, workspace, stream);
}

size_t hif4_gemm_fp8_ws_bytes(int64_t m, int64_t n, int64_t k) {
  if (m == 0 || n == 0 || k == 0) return 0;
  const GemmPlan p = plan_gemm(m, n, k);
  return p.splits == 1 ? 0 : (size_t)p.splits * (size_t)m * (size_t)n * sizeof(float);
}
