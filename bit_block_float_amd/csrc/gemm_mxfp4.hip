// gemm_mxfp4.hip -- Y = X W^T on E2M1 codes with a power-of-two (E8M0) scale per 32
// along K, on gfx950's scaled matrix cores; one W, one W for each group of rows, or
// one Y for each group along K.
//
// Y[i][j] = sum_b sx[i][b] sw[j][b] sum_{t in block b} cx[i][t] cw[j][t].
//
// v_mfma_scale_f32_32x32x64_f8f6f4 (16x16x128 up to 16 rows) on the codes as they
// are. A lane's operand is 32 consecutive values of a row, one block, and the scale
// byte that it gives is that block's. Measured on gfx950: the 4-bit products are
// exact (unlike the 8-bit forms nothing is cut, also where large products of a run
// cancel), and the sums over a block, over the instruction's blocks and onto the
// accumulator are those of fp32: from 64 to 128 products at a time the error stayed
// within 2^-23 of the sum of magnitudes, scale bytes 0 to 254 on either side. So
// results of either type come from the same sums, rounded once for bf16.
//
// The MFMA's first operand is W, so a lane of the result holds one row of Y
// (its column index) and runs of 4 consecutive columns.
#include <algorithm>
#include <type_traits>

#include "gemm_tile_dev.h"
#include "mxfp4_dev.h"

namespace hif4 {

constexpr int kFmtE2M1 = 4;  // cbsz / blgp of the f8f6f4 forms

__device__ __forceinline__ i32x8_t operand(gu32x4_t v) {
  return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}
// 64 values along K; the scale bytes are byte kByte of sa and sb.
template <int kByte>
__device__ __forceinline__ gf32x16_t mfma64(gu32x4_t a, gu32x4_t b, gf32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, kFmtE2M1, kFmtE2M1,
                                                         kByte, (int)sa, kByte, (int)sb);
}
__device__ __forceinline__ gf32x4_t mfma128(gu32x4_t a, gu32x4_t b, gf32x4_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), c, kFmtE2M1, kFmtE2M1,
                                                          0, (int)sa, 0, (int)sb);
}

// This wave's loads but the newest n have landed, its LDS reads are done.
template <int n>
__device__ __forceinline__ void wait_mx4() {
  static_assert(n >= 0 && n < 64, "what the counter holds");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(n) : "memory");
}

struct Mx4Args {
  const uint8_t *x, *xs;
  const uint8_t *w, *ws;
  uint32_t ldx, ldw;  // bytes of a row of codes (a multiple of 64); of scales a 16th
  int64_t m, n;
  int runs;  // of 128 along K (kMx4Depth: of a whole row)
  void* y;
  bool y_bf16;
  int mode;
  uint32_t tiles_m, tiles_n;  // kMx4Rows: tiles_m is the most that the groups can have
  Groups groups;
};

// One tile of Y: its operands from their first row and first run on.
struct Mx4Tile {
  const uint8_t *x, *xs, *w, *ws;
  int mrows, nrows, runs;
  int64_t row0, col0, m;  // in Y, whose rows end at m
  char* y;
};

// Tile t of the product; false: there is none (groups have fewer than their most).
template <int BM, int BN>
__device__ __forceinline__ bool mx4_locate(const Mx4Args& a, uint32_t t, Mx4Tile& tile) {
  constexpr int kShift = BM == 16 ? 4 : BM == 64 ? 6 : BM == 128 ? 7 : 8;
  static_assert(1 << kShift == BM, "a tile's rows");
  int64_t tm, tn, group = 0, k0 = 0;
  int64_t rows_begin = 0, rows_end = a.m;
  tile.runs = a.runs;
  if (a.mode == kMx4Plain) {
    tile_of(t, a.tiles_m, a.tiles_n, tm, tn);
  } else if (a.mode == kMx4Rows) {
    const uint32_t total = group_units(a.groups, kShift) * a.tiles_n;
    if (t >= total) return false;
    t = xcd_order(t, total);
    int e;
    uint32_t before;
    if (!group_unit(a.groups, kShift, t / a.tiles_n, e, before)) return false;
    group_range(a.groups, e, rows_begin, rows_end);
    const uint32_t own = (uint32_t)((rows_end - rows_begin + BM - 1) >> kShift);
    tile_in(t - before * a.tiles_n, own, a.tiles_n, tm, tn);
    group = e;
  } else {
    // each group's tiles over all XCDs: their depth differs from group to group
    const uint32_t per = a.tiles_m * a.tiles_n, e = t / per;
    tile_in(t - e * per, a.tiles_m, a.tiles_n, tm, tn);
    int64_t begin, end;
    group_range(a.groups, (int)e, begin, end);
    // within the row, whatever the offsets say
    k0 = min((int64_t)units_before(a.groups, 7, (int)e), (int64_t)a.runs);
    tile.runs = (int)min((end - begin + 127) >> 7, a.runs - k0);
    group = e;
  }
  tile.row0 = rows_begin + tm * BM;
  tile.col0 = tn * BN;
  tile.m = rows_end;
  if (tile.row0 >= rows_end || tile.col0 >= a.n) return false;
  tile.mrows = (int)min((int64_t)BM, rows_end - tile.row0);
  tile.nrows = (int)min((int64_t)BN, a.n - tile.col0);
  const int64_t wrow = tile.col0 + (a.mode == kMx4Rows ? group * a.n : 0);
  tile.x = a.x + tile.row0 * a.ldx + k0 * 64;
  tile.xs = a.xs + tile.row0 * (a.ldx / 16) + k0 * 4;
  tile.w = a.w + wrow * a.ldw + k0 * 64;
  tile.ws = a.ws + wrow * (a.ldw / 16) + k0 * 4;
  tile.y = reinterpret_cast<char*>(a.y) + (a.mode == kMx4Depth ? group * a.m * a.n * (a.y_bf16 ? 2 : 4) : 0);
  return true;
}

// A tile's operands as buffers: what lies past their last row, or past the last
// row's end, reads as zero.
struct Mx4Buffers {
  __amdgpu_buffer_rsrc_t x, xs, w, ws;
  __device__ __forceinline__ Mx4Buffers(const Mx4Tile& t, uint32_t ldx, uint32_t ldw)
      : x(__builtin_amdgcn_make_buffer_rsrc((void*)t.x, (short)0, (t.mrows - 1) * ldx + t.runs * 64, kRsrc3)),
        xs(__builtin_amdgcn_make_buffer_rsrc((void*)t.xs, (short)0, (t.mrows - 1) * (ldx / 16) + t.runs * 4,
                                             kRsrc3)),
        w(__builtin_amdgcn_make_buffer_rsrc((void*)t.w, (short)0, (t.nrows - 1) * ldw + t.runs * 64, kRsrc3)),
        ws(__builtin_amdgcn_make_buffer_rsrc((void*)t.ws, (short)0, (t.nrows - 1) * (ldw / 16) + t.runs * 4,
                                             kRsrc3)) {}
};

// BM x BN of Y a workgroup, kWM x kWN waves. A stage is 256 values along K (two runs
// of 128): rows of 128 bytes = 8 chunks of 16, chunk c of row r in slot c ^ ((r >> 1)
// & 7), so that the fragment reads of 16 consecutive rows land in distinct bank
// groups, and behind them 16 bytes of scales a row (the stage's 8, and 8 more). kStages
// of them are in LDS, brought by direct-to-LDS buffer loads, 8 rows of codes or 64 of
// scales an instruction, the swizzle applied to the global address. Loads past the last
// stage repeat it, into stages that no one reads; a last stage of one run only has
// bytes in its second half that are not used.
//
// Part `split`: stages [split per_split, (split + 1) per_split) only, the sums to that
// plane of Y as float32 (few tiles and a long K: the parts are added by
// mx4_reduce_kernel in order).
//
// Bound: what the tiles read through L2 (128 x 128: 136 bytes for 32768 operations), and with one or two tiles a CU the latency of their stages in turn. Two
// workgroups a CU: one multiplies while the other waits or stores. 512 x 13824 x 5120 29
// us (2.5 PFLOP/s), 4096 x 4096 x 512 12.2 (1.4); 64 x 64: 32 x 5120 x 5120 8.5 us, both
// gradients of 1001 x 1300 x 640 6.3 to 7.3.
template <int BM, int BN, int kStages>
constexpr int kMx4Lds = kStages * (BM + BN) * (128 + 16) + 1024;  // stages, a sink for idle scale loads
template <int BM, int BN, int kWM, int kWN, int kStages>
__device__ __forceinline__ void mx4_tile(const Mx4Args& a, uint32_t t, int split, int per_split,
                                         char* const lds) {
  constexpr int kWaves = kWM * kWN;
  constexpr int kTM = BM / kWM / 32, kTN = BN / kWN / 32;  // 32 x 32 blocks of a wave
  constexpr int kCodes = (BM + BN) * 128, kStage = kCodes + (BM + BN) * 16;
  constexpr int kGroups = (BM + BN) / 64;  // of 64 rows' scales
  static_assert(kGroups <= kWaves, "one group a wave");

  Mx4Tile tile;
  if (!mx4_locate<BM, BN>(a, t, tile)) return;
  const Mx4Buffers buf(tile, a.ldx, a.ldw);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  const int stages = (tile.runs + 1) / 2;
  const int kb0 = split * per_split, kb1 = min(kb0 + per_split, stages);

  // this wave's scale rows: X's (groups 0 ..), then W's; waves without a group read
  // X's first row into the sink
  const bool has = wave < kGroups, of_x = wave < BM / 64 || !has;
  const __amdgpu_buffer_rsrc_t rs = of_x ? buf.xs : buf.ws;
  const uint32_t soff = !has ? 0u : of_x ? (uint32_t)(wave * 64 + lane) * (a.ldx / 16)
                                         : (uint32_t)((wave - BM / 64) * 64 + lane) * (a.ldw / 16);

  constexpr int kLoads = (BM + BN) / 8 / kWaves;  // of codes, per wave and stage
  constexpr int kXLoads = BM / 8 / kWaves;
  static_assert((BM + BN) % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole loads a wave");
  uint32_t voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const bool x = i < kXLoads;
    const int row = (x ? wave * kXLoads + i : wave * (kLoads - kXLoads) + i - kXLoads) * 8 + (lane >> 3);
    voff[i] = (uint32_t)row * (x ? a.ldx : a.ldw) + (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }
  auto load_stage = [&](int kb, int slot) {
    char* base = lds + slot * kStage;
    const int blk = min(kb, kb1 - 1);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < kXLoads)
        load_lds16(buf.x, base + (wave * kXLoads + i) * 1024, voff[i], blk * 128);
      else
        load_lds16(buf.w, base + BM * 128 + (wave * (kLoads - kXLoads) + i - kXLoads) * 1024, voff[i],
                   blk * 128);
    }
    load_lds16(rs, has ? base + kCodes + wave * 1024 : lds + kStages * kStage, soff, blk * 8);
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
  if (kb0 < kb1) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load_stage(kb0 + s, s);
  }
  int slot = 0;
  for (int kb = kb0; kb < kb1; ++kb) {
    // stage kb has landed for this wave (the loads of the kStages - 2 after it may
    // be in flight); after the barrier for all, and every wave has read the stage
    // that is loaded next
    wait_mx4<(kStages - 2) * (kLoads + 1)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_stage(kb + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
    const char* const stage = lds + slot * kStage;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    gu32x2_t sx[kTM], sw[kTN];  // scale words of the two runs
#pragma unroll
    for (int j = 0; j < kTM; ++j)
      sx[j] = *reinterpret_cast<const gu32x2_t*>(stage + kCodes + (xrow + j * 32) * 16);
#pragma unroll
    for (int i = 0; i < kTN; ++i)
      sw[i] = *reinterpret_cast<const gu32x2_t*>(stage + kCodes + (BM + wrow + i * 32) * 16);
    const char* xs = stage + xrow * 128;
    const char* ws = stage + (BM + wrow) * 128;
    // Run h: lanes 0..31 chunks 4h, 4h + 2, lanes 32..63 the ones behind those; a
    // chunk is a block, its scale the byte of the same number.
    auto run = [&](int h) {
      auto chunk = [&](const char* row, int s) {
        return *reinterpret_cast<const gu32x4_t*>(row + (((4 * h + 2 * s + fhalf) ^ fsw) * 16));
      };
      gu32x4_t fx[kTM][2];
#pragma unroll
      for (int j = 0; j < kTM; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) fx[j][s] = chunk(xs + j * 4096, s);
#pragma unroll
      for (int i = 0; i < kTN; ++i) {
        const gu32x4_t w0 = chunk(ws + i * 4096, 0), w1 = chunk(ws + i * 4096, 1);
#pragma unroll
        for (int j = 0; j < kTM; ++j)
          acc[i][j] = mfma64<0>(w0, fx[j][0], acc[i][j], sw[i][h] >> (8 * fhalf), sx[j][h] >> (8 * fhalf));
#pragma unroll
        for (int j = 0; j < kTM; ++j)
          acc[i][j] = mfma64<2>(w1, fx[j][1], acc[i][j], sw[i][h] >> (8 * fhalf), sx[j][h] >> (8 * fhalf));
      }
    };
    run(0);
    if (2 * kb + 1 < tile.runs) run(1);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  static_assert(kWaves * kStageBytes<false, kTN> <= kMx4Lds<BM, BN, kStages>, "epilogue stage");
  const int64_t row0 = tile.row0 + wm * (BM / kWM), col0 = tile.col0 + wn * (BN / kWN);
  if (a.y_bf16)
    store_tile<true, kTN, kTM>(acc, lds + wave * kStageBytes<true, kTN>, tile.y, row0, col0, tile.m, a.n, lane);
  else
    store_tile<false, kTN, kTM>(acc, lds + wave * kStageBytes<false, kTN>, tile.y + split * a.m * a.n * 4,
                                row0, col0, tile.m, a.n, lane);
}

// One product, or two in one launch, the first with `first` workgroups: few tiles
// leave CUs idle that the second's can have.
template <int BM, int BN, int kWM, int kWN, int kStages>
__global__ __launch_bounds__(kWM* kWN * 64) void mx4_tile_kernel(Mx4Args a, Mx4Args b, uint32_t first,
                                                                 int per_split) {
  __shared__ __attribute__((aligned(1024))) char lds[kMx4Lds<BM, BN, kStages>];
  const bool second = blockIdx.x >= first;
  mx4_tile<BM, BN, kWM, kWN, kStages>(second ? b : a, blockIdx.x - (second ? first : 0u), (int)blockIdx.y,
                                      per_split, lds);
}

// Large products. 256 x 256 of Y a workgroup, 4 waves of 128 x 128 (256 fp32
// accumulators a lane), one workgroup a CU.
//
// A stage is 256 values along K: rows of 128 bytes, whole cache lines, chunk c of 16
// bytes in slot c ^ ((row >> 1) & 7) as above. Two stages are in LDS, each multiplied a
// run (128 values) at a time: while run 0 of stage kb multiplies from registers, run 1
// is read into the other register set; then one barrier, after which no wave needs the
// stage, and stage kb + 2 goes out into it by direct-to-LDS loads while run 1 multiplies
// and run 0 of stage kb + 1 is read. Stages past the end load the last one again, into
// one that no one reads. Where the last stage has one run only, the other's codes are
// loaded as zeros (from beyond the buffers) and its scales taken as 1: with an exit
// between the runs, or a copy of run 0 behind the loop, as tried, the compiler spilled.
//
// Scales come 32 bytes a row, four stages' worth, into a ring of two, one load a stage,
// whose target is chosen without a branch (a branch in the loop lets the compiler move
// products across the step's barrier). Each row's are in a line of their own, and a load
// fetches all 128 bytes of it: 16 bytes a row at a time are half as many bytes from L2 as
// the codes and cost 5%, these half of that.
//
// Bound: the matrix cores at the clock that power allows, and a tile's ends. Measured on
// 57600 x 13824 x 5120, bf16 Y: 1.90 to 1.99 ms (4.2 PFLOP/s); the products alone, from
// registers in as many workgroups, 1.27 ms (6.4, at 1.8 GHz). When it took 2.02 ms, it took
// 1.80 without stores, 1.76 without loads, 1.88 without LDS reads. Loads spread over a
// whole stage, fragments of half a run, rows of 64 bytes in four slots with twice the time
// to land, one barrier more a stage for earlier loads, fragment reads spread over their run
// or in the order of need, and a start of XCDs or CUs at different times (so that not all
// store at once) gave nothing or less. Loads closer together than every other product cost
// 2 to 7%: the path from L2 is the next bound (operands of zeros, which draw little power,
// take 1.54 ms). By depth, a stage takes 1.7 us (5.0 PFLOP/s) and a tile's ends 6 (bf16 Y).
constexpr int kMx4BigSlot = 2 * 256 * 128;
constexpr int kMx4BigRing = 2 * 256 * 32;
constexpr int kMx4BigLds = 2 * kMx4BigSlot + 2 * kMx4BigRing;

__device__ __forceinline__ void mx4_big(const Mx4Args& a, uint32_t t, char* const lds) {
  Mx4Tile tile;
  if (!mx4_locate<256, 256>(a, t, tile)) return;
  const Mx4Buffers buf(tile, a.ldx, a.ldw);
  // (uniform for the compiler, too: it would fetch them from a copy of the arguments lane by lane)
  const uint32_t ldx = __builtin_amdgcn_readfirstlane(a.ldx), ldw = __builtin_amdgcn_readfirstlane(a.ldw);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int stages = (tile.runs + 1) / 2;

  // Loads: instruction i of a wave brings rows 64 wave + 8 (i & 7) .. + 7 of X (i < 8) or
  // W. The swizzle is the same for every other i; 8 i rows go into the scalar offset.
  uint32_t xoff[2], woff[2];
  bool second[2];  // the lane's chunk is of the stage's second run
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t c = (uint32_t)((lane & 7) ^ ((4 * i + (lane >> 4)) & 7));
    xoff[i] = (uint32_t)(wave * 64 + (lane >> 3)) * ldx + c * 16;
    woff[i] = (uint32_t)(wave * 64 + (lane >> 3)) * ldw + c * 16;
    second[i] = c >= 4;
  }
  auto load_part = [&](int kb, int i) {
    char* dst = lds + (kb & 1) * kMx4BigSlot + (i >> 3) * 32768 + wave * 8192 + (i & 7) * 1024;
    const int off = min(kb, stages - 1) * 128;
    const bool half = (tile.runs & 1) && kb >= stages - 1;
    const uint32_t at = half && second[i & 1] ? 0x7FFFFFFFu : (i < 8 ? xoff : woff)[i & 1];
    if (i < 8) load_lds16(buf.x, dst, at, off + (i & 7) * 8 * (int)ldx);
    else load_lds16(buf.w, dst, at, off + (i & 7) * 8 * (int)ldw);
  };
  // A load of scales brings 32 bytes (four stages') of 32 rows, piece p of 16 bytes of row
  // r in slot p ^ ((r >> 3) & 1)
  const uint32_t piece = (uint32_t)((lane & 1) ^ ((lane >> 4) & 1)) * 16;
  const uint32_t xs_off = (uint32_t)(wave * 64 + (lane >> 1)) * (ldx / 16) + piece;
  const uint32_t ws_off = (uint32_t)(wave * 64 + (lane >> 1)) * (ldw / 16) + piece;
  char* const ring = lds + 2 * kMx4BigSlot;
  const int last_group = (stages - 1) >> 2;
  auto load_scale = [&](int kb) {  // kb >= -5
    const int g = ((kb + 1) >> 2) + 1, part = (kb + 1) & 3;
    const bool is_w = part >= 2;
    load_lds16(is_w ? buf.ws : buf.xs,
               ring + (g & 1) * kMx4BigRing + (is_w ? 8192 : 0) + wave * 2048 + (part & 1) * 1024,
               is_w ? ws_off : xs_off,
               min(g, last_group) * 32 + (part & 1) * 2 * (int)(is_w ? ldw : ldx));
  };

  const int frow = lane & 31, fhalf = lane >> 5, fsw = (frow >> 1) & 7;
  const char* const xbase = lds + (wm * 128 + frow) * 128;
  const char* const wbase = lds + 32768 + (wn * 128 + frow) * 128;
  // fragments of a run: blocks of 32 rows 0..3 of X, 4..7 of W, two chunks each
  struct Frags {
    gu32x4_t v[8][2];
  };
  int slot[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) slot[h][e] = ((4 * h + 2 * e + fhalf) ^ fsw) * 16;
  auto read_part = [&](Frags& f, int kb, int h, int p) {  // p = 0..15: block p >> 1, chunk p & 1
    const char* base = ((p >> 1) < 4 ? xbase : wbase) + (kb & 1) * kMx4BigSlot + ((p >> 1) & 3) * 4096;
    f.v[p >> 1][p & 1] = *reinterpret_cast<const gu32x4_t*>(base + slot[h][p & 1]);
  };
  // Scale words, a run each: of the next stage as read, lanes 0..31 a block of 32 rows and
  // lanes 32..63 the one behind it; of this stage, every lane its own row's of each block,
  // its chunks' bytes in bytes 0 and 2.
  gu32x2_t snext[4];
  uint32_t sc[2][8];
  auto read_scale = [&](int kb, int q) {  // blocks 2q and 2q + 1
    const int at = (((kb >> 1) & 1) ^ ((lane >> 3) & 1)) * 16 + (kb & 1) * 8;
    const char* base = ring + ((kb >> 2) & 1) * kMx4BigRing + (q < 2 ? 0 : 8192);
    snext[q] = *reinterpret_cast<const gu32x2_t*>(base + ((q < 2 ? wm : wn) * 128 + (q & 1) * 64 + lane) * 32 + at);
  };

  gf32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // one run (h of stage kb): the products of `cur`, the other run's fragments into
  // `nxt`, and in run 1 the loads of stage kb + 2
  auto run = [&](const Frags& cur, Frags& nxt, int kb, auto h) {
    constexpr int kH = decltype(h)::value;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (c < 16) read_part(nxt, kb + kH, 1 - kH, c);
      if constexpr (kH == 1) {
        if (c == 0) load_scale(kb);
        if ((c & 1) == 1) load_part(kb + 2, c >> 1);
        if (c >= 17 && c < 29 && (c - 17) % 3 == 0) read_scale(kb + 1, (c - 17) / 3);
      }
      const int q = c >> 4, i = (c >> 2) & 3, j = c & 3;
      if (q == 0)
        acc[i][j] = mfma64<0>(cur.v[4 + i][0], cur.v[j][0], acc[i][j], sc[kH][4 + i], sc[kH][j]);
      else
        acc[i][j] = mfma64<2>(cur.v[4 + i][1], cur.v[j][1], acc[i][j], sc[kH][4 + i], sc[kH][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  auto take_scales = [&](int kb) {
    const bool whole = 2 * kb + 1 < tile.runs;
    const uint32_t keep = whole ? ~0u : 0u, one = whole ? 0u : 0x7F7F7F7Fu;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w0 = snext[q].x, w1 = (snext[q].y & keep) | one;
      const auto p0 = __builtin_amdgcn_permlane32_swap(w0, w0, false, false);
      const auto p1 = __builtin_amdgcn_permlane32_swap(w1, w1, false, false);
      sc[0][2 * q] = p0[0] >> (8 * fhalf);
      sc[0][2 * q + 1] = p0[1] >> (8 * fhalf);
      sc[1][2 * q] = p1[0] >> (8 * fhalf);
      sc[1][2 * q + 1] = p1[1] >> (8 * fhalf);
    }
  };
  if (stages > 0) {  // (a group may have no rows, a contraction no depth)
#pragma unroll
    for (int kb = -5; kb < 0; ++kb) load_scale(kb);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) load_part(kb, i);
    asm volatile("s_waitcnt vmcnt(16)" ::: "memory");  // scales and stage 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frags f0, f1;
#pragma unroll
    for (int p = 0; p < 16; ++p) read_part(f0, 0, 0, p);
#pragma unroll
    for (int q = 0; q < 4; ++q) read_scale(0, q);
    for (int kb = 0; kb < stages; ++kb) {
      take_scales(kb);
      run(f0, f1, kb, I0{});
      // stage kb is in registers everywhere, stage kb + 1 has landed
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      run(f1, f0, kb, I1{});
    }
  }
  // every load has landed and every wave has read what it will: the stages are free
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  static_assert(4 * kStageBytes<false, 4> <= kMx4BigLds, "epilogue stage");
  const int64_t row0 = tile.row0 + wm * 128, col0 = tile.col0 + wn * 128;
  if (a.y_bf16)
    store_tile<true, 4, 4>(acc, lds + wave * kStageBytes<true, 4>, tile.y, row0, col0, tile.m, a.n, lane);
  else
    store_tile<false, 4, 4>(acc, lds + wave * kStageBytes<false, 4>, tile.y, row0, col0, tile.m, a.n, lane);
}

__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mx4_big_kernel(Mx4Args a, Mx4Args b, uint32_t first) {
  __shared__ __attribute__((aligned(1024))) char lds[kMx4BigLds];
  const bool second = blockIdx.x >= first;
  mx4_big(second ? b : a, blockIdx.x - (second ? first : 0u), lds);
}

// Y = sum of `splits` float32 planes, in order; 4 elements a thread. Bound: the planes,
// fresh in the caches, and a launch (64 x 5120 in 6: some 4 us of the call's 16.6).
template <bool kBf16>
__global__ __launch_bounds__(256) void mx4_reduce_kernel(const float* __restrict__ parts, int splits,
                                                         int64_t total, void* __restrict__ Y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  const bool vec = (total & 3) == 0;  // whole runs in every plane
  float s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = 0.0f;
  for (int p = 0; p < splits; ++p) {
    const float* src = parts + p * total + i;
    if (vec) {
      const gf32x4_t v = *reinterpret_cast<const gf32x4_t*>(src);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += src[min((int64_t)e, total - 1 - i)];
    }
  }
  store4<kBf16>(Y, i, 0, (int)min((int64_t)4, total - i), vec, s[0], s[1], s[2], s[3]);
}

// Up to 16 kR rows (of a group): bound by reading W once. A wave multiplies 16 columns
// of Y; `parts` waves share them and take K's quads (four runs, 512 values) in turn, and
// their sums meet in LDS in a fixed order; a workgroup has as many sets of such waves as
// its size gives. W goes straight from memory into the MFMA's operand registers: of a
// quad a lane loads four runs' 16 bytes (256 consecutive bytes a row) and the 16 bytes
// of the row's scales for all of them at once, kQuads quads before the first product.
// (A scale word a run, the first way, was as many cache lines again as W itself: one
// row of 13824 x 5120 17.0 us.) Rows past the last or columns past the workgroup's
// repeat the last one and are not stored.
// Measured, one row of 13824 x 5120 (37.6 MB) 8.4 to 9.3 us, 4.0 to 4.5 TB/s with launch
// and the first latency; 96 rows over 32 groups of 5120 x 2048 29 to 33 us, 5.4 to 6.1 TB/s
// of all weights (178 MB, some groups empty, part of W in the 256 MB cache).
template <int kR, int kQuads>
__global__ __launch_bounds__(512) void mx4_skinny_kernel(Mx4Args a, int cols, int parts) {
  __shared__ gf32x4_t sums[8][kR][64];
  static_assert(kR == 1 || kR == 2, "units of 16 or 32 rows");
  constexpr int kShift = kR == 1 ? 4 : 5;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int set = wave / parts, part = wave - set * parts, sets = (int)(blockDim.x >> 6) / parts;
  int64_t row0 = 0, row1 = a.m, wbase = 0;
  const uint32_t unit = blockIdx.x / a.tiles_n;
  if (a.mode == kMx4Rows) {
    int e;
    uint32_t before;
    if (!group_unit(a.groups, kShift, unit, e, before)) return;
    group_range(a.groups, e, row0, row1);
    row0 += (int64_t)(unit - before) << kShift;
    row1 = min(row0 + 16 * kR, row1);
    if (row0 >= row1) return;
    wbase = e * a.n;
  }
  const int64_t n0 = ((int64_t)(blockIdx.x - unit * a.tiles_n) * sets + set) * cols;
  const int64_t n1 = min(n0 + cols, a.n);
  const int rows = (int)(row1 - row0);
  gf32x4_t acc[kR];
#pragma unroll
  for (int j = 0; j < kR; ++j) acc[j] = gf32x4_t{0, 0, 0, 0};
  if (n0 < n1) {  // (else the wave only waits for the others)
    const Mx4Tile tile{a.x + row0 * a.ldx, a.xs + row0 * (a.ldx / 16), a.w + (wbase + n0) * a.ldw,
                       a.ws + (wbase + n0) * (a.ldw / 16), rows, (int)(n1 - n0), a.runs, 0, 0, 0, nullptr};
    const Mx4Buffers buf(tile, a.ldx, a.ldw);
    const int wr = min(r16, tile.nrows - 1);
    const uint32_t wo = wr * a.ldw + kq * 16, wso = wr * (a.ldw / 16);
    uint32_t xo[kR], xso[kR];
#pragma unroll
    for (int j = 0; j < kR; ++j) {
      const int r = min(16 * j + r16, rows - 1);
      xo[j] = r * a.ldx + kq * 16;
      xso[j] = r * (a.ldx / 16);
    }
    auto load = [](__amdgpu_buffer_rsrc_t r, uint32_t lane_off, int off) {
      return __builtin_bit_cast(gu32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, 0));
    };
    const int quads = (a.runs + 3) / 4;
    for (int q0 = part; q0 < quads; q0 += kQuads * parts) {
      gu32x4_t w[kQuads][4], sw[kQuads], x[kQuads][kR][4], sx[kQuads][kR];
#pragma unroll
      for (int u = 0; u < kQuads; ++u) {
        const int q = q0 + u * parts;  // past the end: zeros, or scales that are not used
        if (u > 0 && q >= quads) break;  // uniform
        sw[u] = load(buf.ws, wso, q * 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) w[u][r] = load(buf.w, wo, (4 * q + r) * 64);
#pragma unroll
        for (int j = 0; j < kR; ++j) {
          if (j > 0 && 16 * j >= rows) break;  // uniform
          sx[u][j] = load(buf.xs, xso[j], q * 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) x[u][j][r] = load(buf.x, xo[j], (4 * q + r) * 64);
        }
      }
#pragma unroll
      for (int u = 0; u < kQuads; ++u)
#pragma unroll
        for (int j = 0; j < kR; ++j) {
          if (j > 0 && 16 * j >= rows) break;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (4 * (q0 + u * parts) + r < a.runs)
              acc[j] = mfma128(w[u][r], x[u][j][r], acc[j], sw[u][r] >> (8 * kq), sx[u][j][r] >> (8 * kq));
        }
    }
  }
  if (parts > 1) {
    if (part > 0) {
#pragma unroll
      for (int j = 0; j < kR; ++j) sums[wave][j][lane] = acc[j];
    }
    __syncthreads();
    if (part > 0) return;
    for (int v = 1; v < parts; ++v) {
#pragma unroll
      for (int j = 0; j < kR; ++j) acc[j] += sums[wave + v][j][lane];
    }
  }
  const bool vec = (a.n & 3) == 0 && (cols & 3) == 0 && ((uintptr_t)a.y & 15) == 0;
  const int64_t col = n0 + kq * 4;
#pragma unroll
  for (int j = 0; j < kR; ++j) {
    const int64_t row = row0 + 16 * j + r16;
    if (row < row1 && col < n1) {
      if (a.y_bf16)
        store4<true>(a.y, row * a.n + col, (int)col, (int)n1, vec, acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      else
        store4<false>(a.y, row * a.n + col, (int)col, (int)n1, vec, acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    }
  }
}

enum Mx4Kind { kMx4Skinny, kMx4Skinny2, kMx4Small, kMx4Middle, kMx4Large };
struct Mx4Plan {
  Mx4Kind kind;
  int splits, per_split;  // of K's stages
};
constexpr int64_t kMx4Cus = 256;
static int64_t tiles_in(int64_t v, int64_t tile) { return (v + tile - 1) / tile; }

// Which kernel, from the sizes alone. Measured, bf16 Y, us:
//   m x n x k             16 or 32 rows   64 x 64   128 x 128   256 x 256
//   17 x 5120 x 5120           7.8           8.5       15
//   32 x 2048 x 2048           4.1           5.3        8.2
//   32 x 5120 x 5120           9.5           8.5       15
//   128 x 13824 x 5120                      17         19.6
//   256 x 13824 x 5120                      29         21          31
//   512 x 5120 x 5120                       22         16          31
//   512 x 13824 x 5120                      49         29          32
//   1024 x 5120 x 5120                      38         28          31
//   1024 x 13824 x 5120                     93         56          39
//   2048 x 5120 x 5120                      69         46          33
//   4096 x 4096 x 512                       23         12.2        12.5
//   4096 x 4096 x 2048                      45         26.6        22.7
//   8192 x 8192 x 256                       77         34          39
//   8192 x 8192 x 512                       87         43          46
//   8192 x 8192 x 1024                     112         79          61
// A round of 256 tiles of 256 x 256 costs 4/3 of one of 512 tiles of 128 x 128, from
// some four stages on (below, its ends count, which nothing else on the CU hides).
// Splitting K pays for its second kernel from some 16 stages a part: 64 x 5120 x 5120
// 8.5 us whole, 10.7 in 2; 64 x 5120 x 13824 21 whole, 16.6 in 6, 17 in 3.
static Mx4Plan plan_mx4(int64_t m, int64_t n, int64_t k) {
  const int64_t stages = tiles_in(k, 256);
  const auto tiles = [&](int64_t t) { return tiles_in(m, t) * tiles_in(n, t); };
  // (a grid has fewer than 2^32 threads: 512 for 16 columns, so 2^23 - 1 workgroups)
  if (m <= 16 && n <= (int64_t(1) << 26)) return {kMx4Skinny, 1, (int)stages};
  if (m <= 32 && n <= 4096) return {kMx4Skinny2, 1, (int)stages};
  const int64_t t128 = tiles(128);
  if (stages >= 4 && 4 * tiles_in(tiles(256), kMx4Cus) < 3 * tiles_in(t128, 2 * kMx4Cus))
    return {kMx4Large, 1, (int)stages};
  if (t128 >= kMx4Cus / 2) return {kMx4Middle, 1, (int)stages};
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(2 * kMx4Cus / tiles(64), stages / 16));
  const int64_t per = tiles_in(stages, splits);
  return {kMx4Small, (int)tiles_in(stages, per), (int)per};
}
// The same for rows in groups, by the mean of a group (what is on the host). Measured with
// a skewed choice of groups, bf16 Y, us:
//   groups x mean x n x k     32 rows   64 x 64   128 x 128   256 x 256
//   32 x 3 x 5120 x 2048        32         39         41
//   128 x 4 x 2048 x 1024       30         40         36
//   32 x 8 x 5120 x 2048        45         43         44
//   8 x 8 x 5120 x 5120                    32         38
//   8 x 16 x 5120 x 5120        38         39         40
//   16 x 16 x 2048 x 5120                  22         24
//   32 x 16 x 1536 x 4096                  30         29
//   8 x 16 x 13824 x 5120                  91         81
//   32 x 16 x 5120 x 2048       58         47         45
//   64 x 16 x 2048 x 2048                  40         36
//   128 x 8 x 2048 x 1024                  48         39
//   128 x 16 x 2048 x 1024                 52         42
//   32 x 64 x 5120 x 2048      142         69         50          64
//   128 x 256 x 2048 x 1024               197         97         101
//   32 x 256 x 5120 x 2048                176         97          89
//   8 x 512 x 5120 x 5120                 200        108          82
//   32 x 1024 x 5120 x 2048               571        305         265
// (units of 16 rows instead of 32, 32 x 3 x 5120 x 2048: 35.5: W is read again for the
// second half of a group of more. Few rows a group are one tile each at either size, so the
// small ones pay while the groups' column tiles are some two rounds of the 512 that the CUs
// hold: 32 x 24 of them above are even, 8 x 216 lose from 12 rows a group on.)
static Mx4Plan plan_of(const Mx4Product& p) {
  const int all = (int)tiles_in(p.k, 256);
  if (p.mode == kMx4Plain) return plan_mx4(p.m, p.n, p.k);
  if (p.mode == kMx4Rows) {
    const int64_t mean = tiles_in(p.groups.rows, p.groups.count);
    // (workgroups below 2^23, as above)
    if (mean <= 6 && most_units(p.groups.rows, p.groups.count, 5) * tiles_in(p.n, 16) < (1 << 23))
      return {kMx4Skinny2, 1, all};
    // tiles as if every group ended in the middle of one
    const auto tiles = [&](int64_t t) {
      return (p.groups.rows / t + (p.groups.count + 1) / 2) * tiles_in(p.n, t);
    };
    const bool few = mean <= 16 && p.groups.count * tiles_in(p.n, 64) <= 4 * kMx4Cus;
    if (few || tiles(128) < kMx4Cus / 2) return {kMx4Small, 1, all};
    const bool large = mean >= 256 && mean * p.k >= (1 << 19) &&
                       4 * tiles_in(tiles(256), kMx4Cus) < 3 * tiles_in(tiles(128), 2 * kMx4Cus);
    return {large ? kMx4Large : kMx4Middle, 1, all};
  }
  // K in groups, groups x mean x m x n, us with 128 x 128 and 256 x 256, fp32 Y (bf16): 32 x 64
  // x 2048 x 2048 106 and 110 (83 and 81; Y's bytes 103 and 52), 16 x 256 x 2048 x 5120 134 and
  // 144 (107 and 107; 129 and 65), 16 x 512 x 2048 x 5120 162 and 162 (137 and 126), 16 x 1024 x
  // 2048 x 5120 230 and 194 (205 and 167), 8 x 2048 x 2048 x 5120 187 and 143 (173 and 131), 4 x
  // 512 x 1024 x 1024 7 and 14 (64 x 64: 10).
  const int64_t t256 = p.groups.count * tiles_in(p.m, 256) * tiles_in(p.n, 256);
  if (t256 >= kMx4Cus && p.groups.rows / p.groups.count >= 512) return {kMx4Large, 1, all};
  return {p.groups.count * tiles_in(p.m, 128) * tiles_in(p.n, 128) >= kMx4Cus / 2 ? kMx4Middle : kMx4Small, 1, all};
}

static Mx4Args mx4_args(const Mx4Product& p, int64_t tile) {
  const int shift = tile == 16 ? 4 : tile == 32 ? 5 : tile == 64 ? 6 : tile == 128 ? 7 : 8;
  const int64_t tiles_m = p.mode == kMx4Rows ? most_units(p.groups.rows, p.groups.count, shift) : tiles_in(p.m, tile);
  return Mx4Args{p.x, p.xs, p.w, p.ws, (uint32_t)p.ldx, (uint32_t)p.ldw, p.m, p.n, (int)(p.k / 128), p.y,
                 p.y_bf16, p.mode, (uint32_t)tiles_m, (uint32_t)tiles_in(p.n, tile), p.groups};
}
static uint64_t mx4_tiles(const Mx4Args& a) {
  return (uint64_t)a.tiles_m * a.tiles_n * (a.mode == kMx4Depth ? a.groups.count : 1);
}

// The tile kernels by kind: tile rows and columns, waves both ways, stages.
#define HIF4_MX4_SMALL 64, 64, 2, 2, 4
#define HIF4_MX4_MIDDLE 128, 128, 2, 2, 2

// `b` may be NULL. false: not launched (too many tiles).
static bool launch_mx4_tiles(const Mx4Args& a, const Mx4Args* b, const Mx4Plan& plan, hipStream_t stream) {
  const uint64_t first = mx4_tiles(a), all = first + (b ? mx4_tiles(*b) : 0);
  if (all >= (1ull << 24)) return false;  // a grid has fewer than 2^32 threads
  const dim3 grid((unsigned)all, plan.splits);
#define HIF4_MX4(config, threads)                                                                 \
  hipLaunchKernelGGL((mx4_tile_kernel<config>), grid, dim3(threads), 0, stream, a, b ? *b : a,    \
                     (uint32_t)first, plan.per_split)
  switch (plan.kind) {
    case kMx4Large:
      hipLaunchKernelGGL(mx4_big_kernel, grid, dim3(256), 0, stream, a, b ? *b : a, (uint32_t)first);
      break;
    case kMx4Middle: HIF4_MX4(HIF4_MX4_MIDDLE, 256); break;
    case kMx4Small: HIF4_MX4(HIF4_MX4_SMALL, 256); break;
    default: return false;
  }
#undef HIF4_MX4
  return true;
}

static hipError_t launch_mx4_skinny(const Mx4Product& p, Mx4Kind kind, hipStream_t stream) {
  // Columns of a set of waves: the least that leaves as many sets a CU as 16 would, so
  // that every CU has the same share (of a group, whose number is known on the device
  // only, 16). A wave takes two quads of K at a time where it can, and small workgroups
  // of a group are joined, since each has to find its group first.
  const bool grouped = p.mode == kMx4Rows;
  const int64_t per_cu = tiles_in(p.n, 16 * kMx4Cus), quads = tiles_in(p.k, 512);
  const int cols = grouped ? 16 : (int)tiles_in(p.n, kMx4Cus * per_cu);  // 1 .. 16
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(8, tiles_in(quads, 2)));
  const int sets = grouped ? 8 / parts : 1;
  Mx4Args a = mx4_args(p, kind == kMx4Skinny ? 16 : 32);
  if (!grouped) a.tiles_m = 1;
  a.tiles_n = (uint32_t)tiles_in(p.n, cols * sets);
  const dim3 grid(a.tiles_m * a.tiles_n), block(64 * parts * sets);
  if (kind == kMx4Skinny)
    hipLaunchKernelGGL((mx4_skinny_kernel<1, 2>), grid, block, 0, stream, a, cols, parts);
  else
    hipLaunchKernelGGL((mx4_skinny_kernel<2, 1>), grid, block, 0, stream, a, cols, parts);
  return hipGetLastError();
}
static int64_t mx4_tile_rows(Mx4Kind kind) { return kind == kMx4Small ? 64 : kind == kMx4Large ? 256 : 128; }

}  // namespace hif4

using namespace hif4;

hipError_t hif4_launch_gemm_mxfp4(const Mx4Product& p, void* workspace, hipStream_t stream) {
  const Mx4Plan plan = plan_of(p);
  if (plan.kind <= kMx4Skinny2) return launch_mx4_skinny(p, plan.kind, stream);
  Mx4Args a = mx4_args(p, mx4_tile_rows(plan.kind));
  if (plan.splits == 1)
    return launch_mx4_tiles(a, nullptr, plan, stream) ? hipGetLastError() : hipErrorInvalidValue;
  a.y = workspace;
  a.y_bf16 = false;
  if (!launch_mx4_tiles(a, nullptr, plan, stream)) return hipErrorInvalidValue;
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)tiles_in(p.m * p.n, 1024));
  if (p.y_bf16)
    hipLaunchKernelGGL(mx4_reduce_kernel<true>, grid, dim3(256), 0, stream, (const float*)workspace,
                       plan.splits, p.m * p.n, p.y);
  else
    hipLaunchKernelGGL(mx4_reduce_kernel<false>, grid, dim3(256), 0, stream, (const float*)workspace,
                       plan.splits, p.m * p.n, p.y);
  return hipGetLastError();
}

// Two independent products, in one launch where both take the same tile kernel whole. Where
// they do not, but both are small (64 x 64 tiles cost little more than the kernel for few
// rows, a second launch some 4 us), or as tiles of 128 x 128 fill the CUs once, they share
// one up to a depth of 8 stages each: beyond, a tile's way along K costs more than the
// launch. Both gradients with dY's quantization, us, in one launch and apart, by the depth
// of dX (n / 256; at 8 stages one launch gains 2 us and loses 0.8 at its worst):
//   m x n x k                       one     apart
//   16 x 1024 x 640, 4 stages       9.9     12.3
//   16 x 2048 x 640, 8             11.5     13.1
//   16 x 4096 x 640, 16            18.1     14.9
//   16 x 13824 x 64, 54            22.1     16.3
//   128 x 2048 x 1024, 8           13.8     15.5
//   128 x 4096 x 1024, 16          21.0     18.6
//   128 x 7680 x 1024, 30          31.9     26.0
//   1001 x 1300 x 640 in 5 groups  11.4     14.8 (the products alone)
hipError_t hif4_launch_gemm_mxfp4_two(const Mx4Product& a, const Mx4Product& b, void* workspace,
                                      hipStream_t stream) {
  const Mx4Plan pa = plan_of(a), pb = plan_of(b);
  const auto shallow = [](const Mx4Product& p) {  // (a group of K: in the mean)
    return tiles_in(p.mode == kMx4Depth ? p.k / p.groups.count : p.k, 256) <= 8;
  };
  const bool both = shallow(a) && shallow(b), same = pa.kind == pb.kind && pa.kind >= kMx4Small;
  const bool small = both && pa.kind <= kMx4Small && pb.kind <= kMx4Small;
  const bool once = both && pa.kind <= kMx4Middle && pb.kind <= kMx4Middle &&
                    mx4_tiles(mx4_args(a, 128)) + mx4_tiles(mx4_args(b, 128)) <= 2 * (uint64_t)kMx4Cus;
  if ((same || small || once) && pa.splits == 1 && pb.splits == 1) {
    const Mx4Kind kind = small ? kMx4Small : once ? kMx4Middle : pa.kind;
    const Mx4Args ga = mx4_args(a, mx4_tile_rows(kind)), gb = mx4_args(b, mx4_tile_rows(kind));
    const int most = pa.per_split > pb.per_split ? pa.per_split : pb.per_split;
    if (launch_mx4_tiles(ga, &gb, Mx4Plan{kind, 1, most}, stream)) return hipGetLastError();
  }
  const hipError_t e = hif4_launch_gemm_mxfp4(a, workspace, stream);
  return e != hipSuccess ? e : hif4_launch_gemm_mxfp4(b, workspace, stream);
}

size_t hif4_gemm_mxfp4_ws_bytes(int64_t m, int64_t n, int64_t k) {
  if (m == 0 || n == 0 || k == 0) return 0;
  const Mx4Plan p = plan_mx4(m, n, k);
  return p.splits == 1 ? 0 : (size_t)p.splits * (size_t)m * (size_t)n * sizeof(float);
}
