// Products of e4m3 operands with an fp32 scale for each 128 inputs of an activation row and each 128 x 128 block of a
// weight matrix: dense rows against one matrix, or the pairs of expert bins against their experts' matrices.
//
//   y[i][r] = sum over blocks b: (a_scale[i][b] w_scale[r / 128][b]) * sum over c in b: a[i][c] w[r][c]
//
// Which instruction.  The 8-bit matrix instructions add a lane's products eight at a time with 13 bits under the largest
// one's exponent (1 is lost next to 2^16, among eight neighbouring inputs; between the eights the sum is fp32's): over
// hidden states with loud channels that is 2.5e-5 of the result, 200 times what fp32 sums lose.  e4m3 values are bf16 values
// too, so the kernels here widen them in registers (v_cvt_scalef32_pk_bf16_fp8, exact) and multiply on
// v_mfma_f32_16x16x32_bf16, whose sums are good to 2^-21 of the largest product, at half the rate.
//
// Lane j + 16 g holds 32 of row j's 128 bytes of a block, for both operands, and which 32 does not matter as long
// as both operands take the same: chunks g and g + 4 of 16.  Four instructions add a block up from zero; its sum then
// joins the running one by an fp32 multiply-add with the product of the two scales (arbitrary fp32 numbers: the
// instructions' own scales are powers of two).
#include <algorithm>

#include "f8_device.h"
#include "f8_internal.h"
#include "product_device.h"

namespace qtip {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A lane's 32 values of a block, widened.
struct Wide {
  bf16x8 v[4];
  Wide() = default;
  __device__ explicit Wide(const i32x4 (&c)[2]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t four = (uint32_t)c[i / 4][i % 4];
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(four, 1.0f, true);
      v[i / 2][4 * (i % 2)] = lo[0];
      v[i / 2][4 * (i % 2) + 1] = lo[1];
      v[i / 2][4 * (i % 2) + 2] = hi[0];
      v[i / 2][4 * (i % 2) + 3] = hi[1];
    }
  }
};

// 16 weight rows by 16 activation rows over a block.  Lane j + 16 g gets weight rows 4 g .. 4 g + 3 of row j.
__device__ inline f32x4 multiply_block(const Wide& w, const Wide& a) {
  f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], a.v[i], sum, 0, 0, 0);
  return sum;
}

// U blocks of a row from `at` on, a lane's two chunks of each.  TAIL: they may pass the row's end, `left` bytes away;
// codes behind it are zeros (chunks there read the row's last one again: no branches).
template <int U, bool TAIL>
__device__ inline void load_blocks(const uint8_t* at, int left, i32x4 (&c)[U][2]) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int off = u * kF8Block + h * 64;
      if (!TAIL) {
        c[u][h] = *reinterpret_cast<const i32x4*>(at + off);
      } else {
        const i32x4 v = *reinterpret_cast<const i32x4*>(at + min(off, left - 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) c[u][h][i] = off < left ? v[i] : 0;
      }
    }
}

template <int U, bool TAIL>
__device__ inline void load_scales(const float* row, int first, int blocks, float (&s)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!TAIL) {
      s[u] = row[first + u];
    } else {
      const float v = row[min(first + u, blocks - 1)];
      s[u] = first + u < blocks ? v : 0.0f;
    }
  }
}

// ---- the direct kernel ----------------------------------------------------------------------
// One workgroup: 16 weight rows by up to 16 activation rows, dense; its W waves split the inputs, run by run of U blocks,
// and add their sums through LDS.  Operands go from memory to registers: with few activation rows a call is a
// stream of weights, and the more of them are asked for at once the better.  1 x 4096 x 4096, 16.8 MB of weights:
// 6.1 us, of which about 2 are the launch; 1 x 8192 x 8192: 15.8, 4.2 TB/s.
// TAIL: the rows do not end with a run.
template <int W, bool TAIL>
__global__ __launch_bounds__(W * 64) void direct_kernel(F8MatmulParams p) {
  constexpr int U = 4;
  __shared__ f32x4 red[W][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int j = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16;
  const int blocks = (p.k + kF8Block - 1) / kF8Block;
  int first = wv * U;
  int at = first * kF8Block + g * 16;  // this lane's first byte of the run
  const uint8_t* wc = p.w0 + (size_t)min(n0 + j, p.n - 1) * p.k;
  const float* ws = p.w0_scale + (size_t)(n0 / kF8Block) * blocks;
  const int arow = min(j, p.m - 1);  // rows past the last read it again; never stored
  const uint8_t* ac = p.a + (size_t)arow * p.k;
  const float* as = p.a_scale + (size_t)arow * blocks;
  i32x4 w[U][2] = {};
  if (first < blocks) load_blocks<U, TAIL>(wc + at, p.k - at, w);
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  for (; first < blocks; first += W * U) {
    i32x4 a[U][2];
    float sw[U], sa[U];
    load_scales<U, TAIL>(ws, first, blocks, sw);
    load_blocks<U, TAIL>(ac + at, p.k - at, a);
    load_scales<U, TAIL>(as, first, blocks, sa);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const f32x4 part = multiply_block(Wide(w[u]), Wide(a[u]));
      const float s = sw[u] * sa[u];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(part[i], s, acc[i]);
    }
    at += W * U * kF8Block;
    if (first + W * U < blocks) load_blocks<U, TAIL>(wc + at, p.k - at, w);
  }
  red[wv][lane] = acc;
  __syncthreads();
  if (wv != 0 || j >= p.m) return;
  f32x4 y = red[0][lane];
#pragma unroll
  for (int u = 1; u < W; ++u) y += red[u][lane];
  const float v[4] = {y[0], y[1], y[2], y[3]};
  const int c = n0 + 4 * g;
  if (p.n % 4 != 0) store_odd<4>(p, j, c, v);
  else if (p.out_bf16) store_bf16<4>(p, j, c, v);
  else store_f32<4>(p, j, c, v);
}

// ---- the tiled kernel -----------------------------------------------------------------------
// A workgroup of WM x WN waves computes BM activation rows by BN weight rows (with two matrices BN / 2 rows of each, so
// that a wave holds both factors of its outputs).  A stage is one block of 128 inputs: it goes from memory to LDS
// without passing registers, NST - 1 stages ahead of the one being multiplied; rows and chunks past the operands'
// ends are given an offset past the buffer's range, for which the load writes zeros.
//
// A row's eight 16-byte chunks are stored so that the 16 lanes of an LDS read phase touch 16 different 16-byte
// columns of the banks: see place_of.  The activations' scales of a stage go to LDS beside it, a dword a row; a wave's
// weight rows lie in one 128-row block of a matrix, and its scales of 64 stages stay in a register, a lane each.

// Place of chunk c in LDS row `row`, in 16-byte units, and the other way round.
__device__ inline int place_of(int row, int c) { return c ^ ((row >> 1) & 7); }

// A lane's chunks of an LDS row, for the 8-bit instruction or widened.
template <bool EXACT> struct Fragment {
  Wide v;
  Fragment() = default;
  __device__ explicit Fragment(const i32x4 (&c)[2]) : v(c) {}
  static __device__ f32x4 multiply(const Fragment& w, const Fragment& a) { return multiply_block(w.v, a.v); }
};
template <> struct Fragment<false> {
  i32x8 v;
  Fragment() = default;
  __device__ explicit Fragment(const i32x4 (&c)[2])
      : v{c[0][0], c[0][1], c[0][2], c[0][3], c[1][0], c[1][1], c[1][2], c[1][3]} {}
  static __device__ f32x4 multiply(const Fragment& w, const Fragment& a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
  }
};

// The tile and row block of a workgroup of a dense product: each XCD gets a run of consecutive blocks, as many as any
// other, walked down columns of 8 tiles (the last column may be narrower), so that the blocks running at a time
// share few operand rows.
__device__ inline bool dense_block(int tiles, int row_blocks, int b, int& tile, int& rb) {
  const int total = tiles * row_blocks, each = (total + kXcds - 1) / kXcds;
  const int at = b % kXcds * each + b / kXcds;
  const int column = at / (8 * row_blocks), in = at % (8 * row_blocks);
  const int width = min(8, tiles - column * 8);
  if (b / kXcds >= each || at >= total) return false;
  tile = column * 8 + in % width;
  rb = in / width;
  return true;
}

template <int BM, int BN, int WM, int WN, int NST, int HALVES, bool EXACT, int KG>
__global__ __launch_bounds__(KG * WM * WN * 64) void tiled_kernel(F8MatmulParams p, int tiles, int row_blocks) {
  constexpr int kThreads = WM * WN * 64;              // of a group
  constexpr int kRows = BM + BN;                      // rows of a stage: activations, then weights
  constexpr int kChunks = kF8Block / 16;              // of a row in a stage
  constexpr int kLoads = (kRows * kChunks + kThreads - 1) / kThreads;  // 16-byte loads of a thread and stage
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int FH = FN / HALVES;                     // fragments of one matrix
  constexpr bool kPair = FH % 2 == 0;                 // two fragments side by side: 8 outputs in a lane
  static_assert(BM <= kThreads && FH >= 1 && FH * 16 <= kF8Block && NST >= 2 && NST <= 4, "");
  static_assert(KG == 1 || HALVES == 1, "groups are joined before the results are used");
  constexpr int kWindow = 64 / NST * NST;             // stages whose weight scales a register holds, in whole turns
  constexpr int kCodes = kLoads * kThreads * 16, kStage = kCodes + kThreads * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t c0[KG * kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t c1[KG * kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t c2[NST > 2 ? KG * kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t c3[NST > 3 ? KG * kStage : 16];
  __shared__ uint32_t tops[HALVES == 2 ? BM : 1][WN];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int kg = wave / (WM * WN), wv = wave % (WM * WN);  // group, wave in it
  const int tid = wv * 64 + lane;
  const int wm = wv / WN, wn = wv % WN;
  const int j = lane & 15, g = lane >> 4;

  int tile, rb;
  if (p.offsets) {
    tile_of_block(p, tiles, row_blocks, (int)blockIdx.x, tile, rb);
    if (tile >= tiles) return;
  } else if (!dense_block(tiles, row_blocks, (int)blockIdx.x, tile, rb)) {
    return;
  }
  int expert = 0, start = tile * BM, len = min(BM, p.m - start);
  if (p.offsets && !find_tile(p.offsets, p.E, p.m, BM, tile, expert, start, len)) return;
  const int n0 = rb * (BN / HALVES);
  const int blocks = (p.k + kF8Block - 1) / kF8Block;

  // Row `r` of the weight part of a stage: its matrix and row.  Neighbouring fragments of a wave
  // take rows 8i .. 8i + 3 and 8i + 4 .. 8i + 7, so that a lane's outputs of both are 8 in a row.
  auto weight_row = [&](int r, int& half) {
    const int w = r / (BN / WN), in = r % (BN / WN);
    half = HALVES == 2 ? in / (FH * 16) : 0;
    const int q = in % (FH * 16);
    int col = q;
    if (kPair) col = (q / 32) * 32 + 8 * (q % 16 / 4) + 4 * (q / 16 % 2) + q % 4;
    return n0 + w * (FH * 16) + col;
  };
  // Activation row of tile place i, or -1.
  auto act_row = [&](int i) {
    const int r = tile_row(p, start, len, i);
    return r < 0 ? -1 : (p.offsets ? r / p.a_div : r);
  };

  // Dense activations are addressed from the tile's first row, gathered ones from row 0 (a plan keeps them under
  // 2^30 bytes); their scales, a thirty-second of the codes, likewise.  Weights are addressed from the tile's first
  // row: k is below 2^23, so that 256 rows stay below the buffer's 2^31 bytes.
  const int a_base = p.offsets ? 0 : start;
  const size_t w_base = ((size_t)expert * p.n + n0) * p.k;
  const uint8_t* const a_codes = p.a + (size_t)a_base * p.k;
  const uint8_t* const w0_codes = p.w0 + w_base;
  const uint8_t* const w1_codes = HALVES == 2 ? p.w1 + w_base : nullptr;
  const __amdgpu_buffer_rsrc_t rs = product_rsrc(p.a_scale + (size_t)a_base * blocks);

  // Load i of a thread: LDS row and first byte in the row of the stage.
  auto load_at = [&](int i, int& r, int& byte) {
    const int slot = i * kThreads + tid;
    r = slot / kChunks;
    byte = place_of(r, slot % kChunks) * 16;  // its own inverse
  };
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    int r, byte;
    load_at(i, r, byte);
    if (r < BM) {
      const int row = act_row(r);
      off[i] = row < 0 ? kNoRow : (uint32_t)((size_t)(row - a_base) * p.k) + byte;
    } else {
      int half;
      const int row = weight_row(r - BM, half);
      off[i] = r < kRows && row < p.n ? (uint32_t)((size_t)(row - n0) * p.k) + byte : kNoRow;
    }
  }
  const int scale_row = tid < BM ? act_row(tid) : -1;
  const uint32_t scale_off = scale_row < 0 ? kNoRow : (uint32_t)((size_t)(scale_row - a_base) * blocks * 4);
  // Loads [i0, i1) of stage s's codes; its scales.
  auto issue_codes = [&](uint8_t* dst, int s, int i0, int i1) __attribute__((always_inline)) {
    const int block = s * KG + kg, so = min(block, blocks) * kF8Block;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < i0 || i >= i1) continue;
      // chunks past the row's end, and stages past the last
      int r, byte;
      load_at(i, r, byte);
      const uint32_t o = block * kF8Block + byte < p.k ? off[i] : kNoRow;
      lds_void* at = (lds_void*)(dst + kg * kStage + (i * kThreads + wv * 64) * 16);
      const int row = (i * kThreads + wv * 64) / kChunks;  // a wave's load is of eight rows of one fragment
      const bool of_a = (i + 1) * kThreads <= BM * kChunks || (i * kThreads < BM * kChunks && row < BM);
      int half = 0;
      if (HALVES == 2) weight_row(row - BM, half);
      const uint8_t* base = of_a ? a_codes : HALVES == 2 && half ? w1_codes : w0_codes;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(product_rsrc(base), at, 16, o, so, 0, 0);
    }
  };
  auto issue_scales = [&](uint8_t* dst, int s) __attribute__((always_inline)) {
    const int block = s * KG + kg;
    const uint32_t o = block < blocks ? scale_off : kNoRow;
    lds_void* at = (lds_void*)(dst + kg * kStage + kCodes + wv * 256);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, at, 4, o, min(block, blocks) * 4, 0, 0);
  };

  // The weights' scales of the group's stages from s on, a lane each; 0 for stages past the last.
  const int wb = min(n0 + wn * (FH * 16), p.n - 1) / kF8Block;
  const size_t ws_row = ((size_t)expert * ((p.n + kF8Block - 1) / kF8Block) + wb) * blocks;
  float ws[HALVES];
  auto load_window = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const int block = (s + lane) * KG + kg;
      const float v = (h ? p.w1_scale : p.w0_scale)[ws_row + min(block, blocks - 1)];
      ws[h] = block < blocks ? v : 0.0f;
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int a_row = wm * (BM / WM) + j, w_row = BM + wn * (BN / WN) + j;
  const int col0 = place_of(j, g) * 16, col1 = place_of(j, g + 4) * 16;  // rows 16 apart have the same order of places
  struct Raw { i32x4 c[2]; };
  auto read = [&](const uint8_t* cur, int row) __attribute__((always_inline)) {
    const uint8_t* at = cur + row * kF8Block;
    return Raw{{*reinterpret_cast<const i32x4*>(at + col0), *reinterpret_cast<const i32x4*>(at + col1)}};
  };
  // The sums of a row of fragments join the running ones while the next row is multiplied, also from a stage to the next.
  f32x4 old[FN];
  float old_scale[HALVES];
#pragma unroll
  for (int b = 0; b < FN; ++b) old[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < HALVES; ++h) old_scale[h] = 0.0f;
  auto add_old = [&](int a, int b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(old[b][i], old_scale[b / FH], acc[a][b][i]);
  };
  // One stage.  Before it is read, its loads have to have arrived (the stages after it stay in flight) and every
  // wave has to have read the stage whose place the next load takes.  A large tile's next loads go out one by one
  // between the first half's products: all at once they hold up the wave, and the products behind them, until the address
  // unit has taken them (4096 x 8192 x 8192: 241 us, at once 257).  A small one waits for memory and asks at once.
  constexpr bool kEarly = BM <= 64;
  // N: fragments of rows that are multiplied, the others hold no row.
  auto stage = [&](auto fragments, const uint8_t* buf, uint8_t* next, int s) __attribute__((always_inline)) {
    constexpr int N = decltype(fragments)::value;
    constexpr int kIssue = N * FN > 1 ? N * FN / 2 : 1;
    wait_loads<(NST - 2) * (kLoads + 1)>();
    wave_barrier();
    if (kEarly) issue_codes(next, s + NST - 1, 0, kLoads);
    const uint8_t* cur = buf + kg * kStage;
    const float* scales = reinterpret_cast<const float*>(cur + kCodes) + a_row;
    Fragment<EXACT> fw[FN], fa(read(cur, a_row).c);
    float sa = scales[0], sw[HALVES];
    if (!EXACT) __builtin_amdgcn_sched_barrier(0);  // the products begin as the fragments come
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      fw[b] = Fragment<EXACT>(read(cur, w_row + 16 * b).c);
      if (!EXACT) __builtin_amdgcn_sched_barrier(0);
    }
    issue_scales(next, s + NST - 1);
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
      sw[h] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ws[h]), s % kWindow));
#pragma unroll
    for (int b = 0; b < FN; ++b) add_old(N - 1, b);
    if (!EXACT) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int a = 0; a < N; ++a) {
      const int next_row = 16 * (a + 1 < N ? a + 1 : a);
      const Raw a_next = read(cur, a_row + next_row);
      const float sa_next = scales[next_row];
      if (!EXACT) __builtin_amdgcn_sched_barrier(0);
      f32x4 sum[FN];
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        sum[b] = Fragment<EXACT>::multiply(fw[b], fa);
        if (a > 0) add_old(a - 1, b);
        const int step = a * FN + b;
        if (!kEarly) issue_codes(next, s + NST - 1, step * kLoads / kIssue, (step + 1) * kLoads / kIssue);
        if (!EXACT) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int b = 0; b < FN; ++b) old[b] = sum[b];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) old_scale[h] = sa * sw[h];
      fa = Fragment<EXACT>(a_next.c);
      sa = sa_next;
      if (EXACT) __builtin_amdgcn_sched_barrier(0);
    }
  };

  load_window(0);
#pragma unroll
  for (int s = 0; s < NST - 1; ++s) {
    uint8_t* dst = s == 0 ? c0 : s == 1 ? c1 : c2;
    issue_scales(dst, s);
    issue_codes(dst, s, 0, kLoads);
  }
  // Whole turns: the stages past the last one add zeros.
  const int stages = (blocks + KG - 1) / KG;
  auto run = [&](auto fragments) __attribute__((always_inline)) {
    for (int s = 0; s < stages; s += NST) {
      if (s > 0 && s % kWindow == 0) load_window(s);
      if (NST == 2) {
        stage(fragments, c0, c1, s);
        stage(fragments, c1, c0, s + 1);
      } else if (NST == 3) {
        stage(fragments, c0, c2, s);
        stage(fragments, c1, c0, s + 1);
        stage(fragments, c2, c1, s + 2);
      } else {
        stage(fragments, c0, c3, s);
        stage(fragments, c1, c0, s + 1);
        stage(fragments, c2, c1, s + 2);
        stage(fragments, c3, c2, s + 3);
      }
    }
#pragma unroll
    for (int b = 0; b < FN; ++b) add_old(decltype(fragments)::value - 1, b);
  };
  // A wave whose second half of rows is empty (an expert's last tile) leaves it out.
  constexpr bool kHalf = FM == 2 || (FM > 2 && !EXACT);
  if (kHalf && len <= wm * (BM / WM) + BM / WM / 2) run(Step<(FM + 1) / 2>());
  else run(Step<FM>());
  __builtin_amdgcn_s_waitcnt(0);  // no load to LDS outlives the workgroup
  if constexpr (KG > 1) {
    static_assert(KG <= 2 && BM * BN * 4 <= KG * kStage, "the second group's sums go through the first stage's place");
    f32x4* sums = reinterpret_cast<f32x4*>(c0) + tid;
    __syncthreads();
    if (kg == 1) {
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b) sums[(a * FN + b) * kThreads] = acc[a][b];
    }
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b) acc[a][b] += sums[(a * FN + b) * kThreads];
  }

  // Lane j + 16 g of fragment (a, b): activation row 16 a + j, weight rows 4 g .. 4 g + 3 of b.
  constexpr int kSpan = kPair ? 8 : 4;
  auto result = [&](int a, int b, float (&v)[kSpan]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      v[i] = acc[a][b + i / 4][i % 4];
      if (HALVES == 2) v[i] = swiglu(v[i], acc[a][(HALVES - 1) * FH + b + i / 4][i % 4]);
    }
  };
  const int col = n0 + wn * (FH * 16) + (kPair ? 8 * g : 4 * g);  // of fragment 0
  if (HALVES == 2 && p.out_scale) {
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      uint32_t top = 0;
#pragma unroll
      for (int b = 0; b < FH; b += kPair ? 2 : 1) {
        float v[kSpan];
        result(a, b, v);
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
          acc[a][b + i / 4][i % 4] = v[i];
          top = max(top, f8_bits(v[i]) & 0x7fffffffu);
        }
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      if (g == 0) tops[a_row + 16 * a][wn] = top;
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      const int r = tile_row(p, start, len, a_row + 16 * a);
      if (r < 0) continue;
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < WN; ++w) top = max(top, tops[a_row + 16 * a][w]);
      const F8Scale s(top, false);
#pragma unroll
      for (int b = 0; b < FH; b += kPair ? 2 : 1) {
        float v[kSpan];
#pragma unroll
        for (int i = 0; i < kSpan; ++i) v[i] = acc[a][b + i / 4][i % 4];
        uint32_t codes[kSpan / 4];
        f8_codes(v, s, codes);
        uint8_t* d = reinterpret_cast<uint8_t*>(p.out) + (size_t)r * p.n + col + 16 * b;
        if (kPair) *reinterpret_cast<uint2*>(d) = make_uint2(codes[0], codes[kSpan / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(d) = codes[0];
      }
      if (wn == 0 && g == 0) p.out_scale[(size_t)r * (p.n / kF8Block) + rb] = s.scale;
    }
    return;
  }
  auto write = [&](auto store) __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      const int r = tile_row(p, start, len, a_row + 16 * a);
#pragma unroll
      for (int b = 0; b < FH; b += kPair ? 2 : 1) {
        float v[kSpan];
        result(a, b, v);
        if (r >= 0) store(r, col + 16 * b, v);
      }
    }
  };
  if (p.n % kSpan != 0)
    write([&](int r, int c, const float (&v)[kSpan]) { store_odd<kSpan>(p, r, c, v); });
  else if (p.out_bf16)
    write([&](int r, int c, const float (&v)[kSpan]) { store_bf16<kSpan>(p, r, c, v); });
  else
    write([&](int r, int c, const float (&v)[kSpan]) { store_f32<kSpan>(p, r, c, v); });
}

// Tiles of at most bm rows there can be: an expert's last tile may be partly filled, at most one more per expert
// that has pairs.  64 bits: m and n go up to 2^31 - 1.
int64_t most_tiles(const F8MatmulParams& p, int bm) {
  if (p.offsets) return p.m / bm + (p.m < p.E ? p.m : p.E);
  return ((int64_t)p.m + bm - 1) / bm;
}

template <int W>
hipError_t launch_direct(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  const int64_t grid = ((int64_t)p.n + 15) / 16;
  if (grid * (W * 64) > kMostThreads) return hipErrorInvalidConfiguration;
  if (!launch) return hipSuccess;
  if (p.k % (4 * kF8Block) == 0)
    hipLaunchKernelGGL((direct_kernel<W, false>), dim3((unsigned)grid), dim3(W * 64), 0, stream, p);
  else
    hipLaunchKernelGGL((direct_kernel<W, true>), dim3((unsigned)grid), dim3(W * 64), 0, stream, p);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NST, int HALVES, bool EXACT, int KG = 1>
hipError_t launch_tiled(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  const int64_t tiles = most_tiles(p, BM);
  const int64_t row_blocks = ((int64_t)p.n + BN / HALVES - 1) / (BN / HALVES);
  const int64_t grid = p.offsets ? (tiles + kXcds - 1) / kXcds * kXcds * row_blocks
                                 : (tiles * row_blocks + kXcds - 1) / kXcds * kXcds;
  constexpr int threads = KG * WM * WN * 64;
  if (grid * threads > kMostThreads) return hipErrorInvalidConfiguration;
  if (!launch) return hipSuccess;
  hipLaunchKernelGGL((tiled_kernel<BM, BN, WM, WN, NST, HALVES, EXACT, KG>), dim3((unsigned)grid), dim3(threads), 0,
                     stream, p, (int)tiles, (int)row_blocks);
  return hipGetLastError();
}

// Which kernel and tile.  Large tiles read the operands less often, small ones make more workgroups; below about one
// workgroup a CU a second group of waves that takes every other stage hides the waits instead.  bf16 results of tiles
// that wait for the matrix instructions come from the 8-bit ones, all others from the exact ones (see the top).
// Times in us at m x n x k, or, unless a line says otherwise, of a 256-expert, top-6 layer of 4096 x 2048, each side of
// a border:
//   direct up to 16 rows  1 x 4096 x 4096 direct 6.1, 16 x 64 tiles 13.0; 17 rows 10.0, 32 x 64 8.9
//   256 x 256             where tiles of 128 x 256 take a second turn on 256 CUs: 2500 x 4096 x 2048 (320 of those) 27.4,
//                         128 x 256 36.1; 1792 x 8192 x 4096 (448) 54.3, 64.5; 2048 x 4096 x 4096 (256) 46, 35.7
//   128 x 256 from 200    three stages: 1500 x 5120 x 4096 (240) 34.1, 128 x 128 39.3; 1024 x 4096 x 4096 (128) 29.3, two
//                         groups of 64 x 128 25.0; 1024 x 8192 x 2048 (256) 22.2, 128 x 128 23.8, 64 x 128 28.1; of 512
//                         inputs 4096 x 2048 x 512 (256) 11.3, 128 x 128 10.6
//   128 x 128 from 400    (these, and exact)
//   64 x 128 from 160     1000 x 2056 x 4096 (272) 23.0, 32 x 128 25.8, two groups 34; two groups up to 256: 512 x 4096 x
//                         4096 (256) 16.1, 32 x 128 20.3, one group 21.4; 683 x 2056 x 4064, exact, (187) 24.4,
//                         32 x 128 29.3
//   32 x 128 from 160     256 x 4096 x 4096 (256) 12.1, 32 x 64 16.4; 128 x 4096 x 4096 (128) 14.5, 9.7; two groups up to
//                         256: 300 x 2056 x 4064 (170) 16.6, one 19.0
//   stages of two groups  512 x 4096 x 4096 three 16.1, two 17.7; exact 683 x 2056 x 4064 three 28, two 24.4
//   exact, large          4096 x 8192 x 8192 128 x 128 493, 64 x 128 570; the 8-bit instructions 240 (256 x 256)
// These rules ask for workgroups, not whether m and n fill a tile.  Where one of the two is small and the other very
// large they take too large a tile: 32 x 129280 x 7168 256 x 256 194, 128 x 256 161, 32 x 128 180, exact 128 x 128 223,
// 32 x 128 185; 128 x 129280 x 7168 256 x 256 220, 128 x 256 200; 65536 x 32 x 4096 256 x 256 74, 128 x 128 69.
// Expert passes take the largest of these tiles that their pairs an expert fill and that makes enough workgroups, both
// by the average (the bins are on the device; skewed routing makes more tiles of the same pairs):
//   gate+up               24 pairs an expert 32 rows 776, 64 rows 889; 48 pairs 1130, 959; 96 pairs 64 rows 1582, 128 rows
//                         1213; workgroups of 128 rows: 128 57, 64 rows 47 (1 expert, 1024 pairs); 192 57, 64 rows 84;
//                         of 64 rows: 16 15.3, 32 rows 11.0 (1 expert, 100 pairs of 1024 x 1024); 256 47, 32 rows 48
//                         8-bit, 128 rows: 128 workgroups 38.5, exact 47; 8 13.2, exact 11.0; 24000 pairs of 24 experts
//                         in three stages 532, in two 616, exact 814, 256 rows 438; workgroups of 256 rows: 96 50, 128
//                         rows 33 (1 expert, 3000 pairs of 1024 x 4096); 128 65, 128 rows 75 (8 experts, 2000 pairs)
//                         up to 128 workgroups of 32 rows four stages: 6 pairs (96) 29.8, two 38.2; 24 pairs (384) 78, 73
//   down                  24 pairs 32 rows 458, 64 rows 461; 48 pairs 64 rows 490, 128 rows 514; 96 pairs 664, 574;
//                         96 pairs 128 rows 574, 256 rows 609; 192 pairs 970, 717; workgroups of 256 rows: 96 16.1, 128 rows
//                         13.8 (8 experts, 6000 pairs of 512 x 1024); 128 35.5, 128 rows 44; of 128 rows: 8 15.1, 32 x 64
//                         7.4 (1 expert, 100 pairs of 1024 x 1024); 256 26.5, 64 rows 27.4; of 32 x 128: 128 12.9, 32 x 64 of
//                         two groups 10.5 (8 experts, 120 pairs of 2048 x 2048); 192 13.3, 16.8
//                         8-bit: 83 pairs 128 x 256 57.5, 128 x 128 63.7 (24 experts, 2000 pairs); 1024 inputs 18.1, 18.8 (8
//                         experts, 1100 pairs of 4096), 512 inputs 26.4, 24.0 (64 experts, 5400 pairs of 2048); 128
//                         workgroups of 128 x 128 20.3, exact 64 x 128 23.8 (8 experts, 900 pairs of 2048 x 2048)
// Without `launch` it says whether the launch could be made.
template <bool EXACT>
hipError_t launch_dense(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  constexpr int kDeep = EXACT ? 2 : 3;  // stages of two groups of waves, one workgroup a CU
  auto groups = [&](int64_t bm, int64_t bn) { return (p.m + bm - 1) / bm * ((p.n + bn - 1) / bn); };
  if constexpr (!EXACT) {
    if (groups(128, 256) > 256) return launch_tiled<256, 256, 2, 4, 2, 1, false>(p, stream, launch);
    if (groups(128, 256) >= 200 && p.k > 4 * kF8Block)
      return launch_tiled<128, 256, 2, 4, 3, 1, false>(p, stream, launch);
  }
  if (groups(128, 128) >= 400) return launch_tiled<128, 128, 2, 2, 2, 1, EXACT>(p, stream, launch);
  if (groups(64, 128) > 256) return launch_tiled<64, 128, 1, 4, 2, 1, EXACT>(p, stream, launch);
  if (groups(64, 128) >= 160) return launch_tiled<64, 128, 2, 2, kDeep, 1, EXACT, 2>(p, stream, launch);
  if (groups(32, 128) > 256) return launch_tiled<32, 128, 1, 4, 2, 1, EXACT>(p, stream, launch);
  if (groups(32, 128) >= 160) return launch_tiled<32, 128, 1, 4, kDeep, 1, EXACT, 2>(p, stream, launch);
  return launch_tiled<32, 64, 1, 2, 4, 1, EXACT, 2>(p, stream, launch);
}

hipError_t choose(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  if (!p.offsets) {
    if (p.m <= 16) return launch_direct<8>(p, stream, launch);
    return p.out_bf16 ? launch_dense<false>(p, stream, launch) : launch_dense<true>(p, stream, launch);
  }
  const int64_t fill = ((int64_t)p.m + p.E - 1) / p.E;  // pairs an expert gets on average
  auto groups = [&](int64_t bm, int64_t bn) {
    return std::min(p.m, p.E) * ((fill + bm - 1) / bm) * ((p.n + bn - 1) / bn);
  };
  if (p.w1) {
    if (p.out_bf16 && fill > 160 && groups(256, 128) >= 128)
      return launch_tiled<256, 256, 2, 4, 2, 2, false>(p, stream, launch);
    if (p.out_bf16 && fill > 64 && groups(128, 128) >= 128)
      return launch_tiled<128, 256, 2, 4, 3, 2, false>(p, stream, launch);
    if (fill > 64 && groups(128, 128) > 160) return launch_tiled<128, 256, 2, 4, 2, 2, true>(p, stream, launch);
    if (fill > 28 && groups(64, 128) > 160) return launch_tiled<64, 256, 1, 4, 2, 2, true>(p, stream, launch);
    if (groups(32, 128) > 128) return launch_tiled<32, 256, 1, 4, 2, 2, true>(p, stream, launch);
    return launch_tiled<32, 256, 1, 4, 4, 2, true>(p, stream, launch);
  }
  if (p.out_bf16 && fill > 160 && groups(256, 256) >= 128)
    return launch_tiled<256, 256, 2, 4, 2, 1, false>(p, stream, launch);
  if (p.out_bf16 && fill > 64 && groups(128, 128) >= 128)
    return p.k > 4 * kF8Block ? launch_tiled<128, 256, 2, 4, 3, 1, false>(p, stream, launch)
                              : launch_tiled<128, 128, 2, 2, 2, 1, false>(p, stream, launch);
  if (fill > 64 && groups(128, 128) > 160) return launch_tiled<128, 128, 2, 2, 2, 1, true>(p, stream, launch);
  if (fill > 28 && groups(64, 128) > 160) return launch_tiled<64, 128, 1, 4, 2, 1, true>(p, stream, launch);
  if (groups(32, 128) >= 160) return launch_tiled<32, 128, 1, 4, 2, 1, true>(p, stream, launch);
  return launch_tiled<32, 64, 1, 2, 4, 1, true, 2>(p, stream, launch);
}

}  // namespace

hipError_t launch_f8_matmul(const F8MatmulParams& p, hipStream_t stream) { return choose(p, stream, true); }

bool f8_matmul_fits(const F8MatmulParams& p) { return choose(p, nullptr, false) == hipSuccess; }

}  // namespace qtip
