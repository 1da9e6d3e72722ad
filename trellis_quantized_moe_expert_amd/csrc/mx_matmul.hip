// Products of MXFP4 operands on the scaled matrix instructions (v_mfma_scale_f32_16x16x128_f8f6f4):
// dense rows against one matrix, or the pairs of expert bins against their experts' matrices.
//
// One instruction multiplies 16 weight rows by 16 activation rows over 128 inputs.  Lane j + 16 g
// holds row j's codes of one block of 32 inputs (16 bytes) and that block's scale byte, for both
// operands; which four blocks an instruction takes does not matter as long as both operands take
// the same.  So lane group g reads the 64 contiguous bytes of blocks 4g .. 4g + 3 of each run of 16
// blocks and feeds four instructions with them, and one dword holds the lane's four scales (the
// instruction picks its byte).
#include "mx_internal.h"
#include "product_device.h"
#include "qtip_internal.h"

#include <cmath>

namespace qtip {

namespace {

constexpr int kFp4 = 4;  // the operand format of the f8f6f4 instructions: e2m1

template <int SEL>
__device__ inline f32x4 mfma_fp4(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  const i32x8 a8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8{b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, kFp4, kFp4, SEL, sa, SEL, sb);
}

// ---- the direct kernel ----------------------------------------------------------------------
// One workgroup: 16 weight rows (of both matrices where there are two) by MB * 16 activation rows;
// its W waves split the inputs, run by run of 512, and add their sums through LDS.  Operands go from
// memory to registers: with few activation rows a call is a stream of weights, and the more of them
// are asked for at once the better.  Bound by those loads: 6 pairs of a 4096 x 2048 gate+up pass, 53.5 MB
// of weights, 12.7 to 13.8 us (4.2 TB/s; 11.3 at the copy rate); 1 x 4096 x 4096, 8.9 MB, 4.0 us, of which
// about 2 are the launch.
// TAIL: the rows do not end with a run.
template <int MB, int HALVES, int W, bool TAIL>
__global__ __launch_bounds__(W * 64, MB * HALVES == 1 ? 6 : MB * HALVES == 2 ? 5 : 2) void direct_kernel(
    MxMatmulParams p) {
  __shared__ f32x4 red[W][HALVES * MB][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int j = lane & 15, g = lane >> 4;
  const int row_blocks = (p.n + 15) >> 4;
  const int tile = (int)blockIdx.x / row_blocks;
  const int n0 = ((int)blockIdx.x - tile * row_blocks) * 16;
  int expert = 0, start = tile * MB * 16, len = min(MB * 16, p.m - start);
  if (p.offsets && !find_tile(p.offsets, p.E, p.m, MB * 16, tile, expert, start, len)) return;

  const size_t row_codes = (size_t)p.blocks * kMxBlockBytes;
  const size_t wrow = (size_t)expert * p.n + min(n0 + j, p.n - 1);
  const uint8_t* wc[2] = {p.w0 + wrow * row_codes, HALVES == 2 ? p.w1 + wrow * row_codes : nullptr};
  const uint8_t* ws[2] = {p.w0_scale + wrow * p.blocks, HALVES == 2 ? p.w1_scale + wrow * p.blocks : nullptr};

  // Four blocks of a row from block `first` on, and their scales; zero codes past the row's end.
  auto load = [&](const uint8_t* codes, const uint8_t* scales, int first, i32x4 (&c)[4], int& s) {
    typedef uint32_t __attribute__((aligned(1))) u32_any;
    if (!TAIL) {
#pragma unroll
      for (int st = 0; st < 4; ++st)
        c[st] = *reinterpret_cast<const i32x4*>(codes + (size_t)(first + st) * kMxBlockBytes);
      s = (int)*reinterpret_cast<const u32_any*>(scales + first);
    } else {
      s = 0;
#pragma unroll
      for (int st = 0; st < 4; ++st) {  // blocks past the end read the last one again; no branches
        const bool in = first + st < p.blocks;
        const int at = min(first + st, p.blocks - 1);
        const i32x4 v = *reinterpret_cast<const i32x4*>(codes + (size_t)at * kMxBlockBytes);
        const int scale = scales[at];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[st][i] = in ? v[i] : 0;
        s |= (in ? scale : 127) << (8 * st);
      }
    }
  };
  int first = wv * 16 + 4 * g;
  i32x4 w[HALVES][4];
  int sw[HALVES];
  if (wv * 16 < p.blocks) {  // before the activation rows are looked up
#pragma unroll
    for (int h = 0; h < HALVES; ++h) load(wc[h], ws[h], first, w[h], sw[h]);
  }

  const uint8_t* ac[MB];
  const uint8_t* as[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int r = tile_row(p, start, len, 16 * b + j);
    const size_t arow = (size_t)(r < 0 ? 0 : r / p.a_div);  // rows past the tile read row 0; never stored
    ac[b] = p.a + arow * row_codes;
    as[b] = p.a_scale + arow * p.blocks;
  }
  f32x4 acc[HALVES][MB];
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[h][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int run = wv; run * 16 < p.blocks; run += W) {
    i32x4 a[MB][4];
    int sa[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) load(ac[b], as[b], first, a[b], sa[b]);
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        acc[h][b] = mfma_fp4<0>(w[h][0], a[b][0], acc[h][b], sw[h], sa[b]);
        acc[h][b] = mfma_fp4<1>(w[h][1], a[b][1], acc[h][b], sw[h], sa[b]);
        acc[h][b] = mfma_fp4<2>(w[h][2], a[b][2], acc[h][b], sw[h], sa[b]);
        acc[h][b] = mfma_fp4<3>(w[h][3], a[b][3], acc[h][b], sw[h], sa[b]);
      }
    first += W * 16;
    if ((run + W) * 16 < p.blocks) {
#pragma unroll
      for (int h = 0; h < HALVES; ++h) load(wc[h], ws[h], first, w[h], sw[h]);
    }
  }
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int b = 0; b < MB; ++b) red[wv][h * MB + b][lane] = acc[h][b];
  __syncthreads();
  // Lane j + 16 g of fragment b holds weight rows n0 + 4g .. + 3 of activation row 16 b + j.
  for (int q = threadIdx.x; q < MB * 64; q += W * 64) {
    const int b = q >> 6, ln = q & 63;
    const int r = tile_row(p, start, len, 16 * b + (ln & 15));
    if (r < 0) continue;
    f32x4 y[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      y[h] = red[0][h * MB + b][ln];
#pragma unroll
      for (int u = 1; u < W; ++u) y[h] += red[u][h * MB + b][ln];
    }
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = y[0][i];
      if (HALVES == 2) v[i] = swiglu(v[i], y[HALVES - 1][i]);
    }
    const int c = n0 + 4 * (ln >> 4);
    if (p.n % 4 != 0) store_odd<4>(p, r, c, v);
    else if (p.out_bf16) store_bf16<4>(p, r, c, v);
    else store_f32<4>(p, r, c, v);
  }
}

template <int MB, int HALVES, int W>
hipError_t launch_direct(const MxMatmulParams& p, hipStream_t stream, bool launch) {
  int64_t tiles = ((int64_t)p.m + MB * 16 - 1) / (MB * 16);  // 64 bits: m and n go up to 2^31 - 1
  // an expert's last tile may be partly filled: at most one more per expert that has pairs
  if (p.offsets) tiles = p.m / (MB * 16) + (p.m < p.E ? p.m : p.E);
  const int64_t grid = tiles * (((int64_t)p.n + 15) / 16);
  if (grid * (W * 64) > kMostThreads) return hipErrorInvalidConfiguration;
  if (!launch) return hipSuccess;
  if (p.blocks % 16 == 0)
    hipLaunchKernelGGL((direct_kernel<MB, HALVES, W, false>), dim3((unsigned)grid), dim3(W * 64), 0, stream, p);
  else
    hipLaunchKernelGGL((direct_kernel<MB, HALVES, W, true>), dim3((unsigned)grid), dim3(W * 64), 0, stream, p);
  return hipGetLastError();
}

// ---- the tiled kernel -----------------------------------------------------------------------
// A workgroup of WM x WN waves computes BM activation rows by BN weight rows (with two matrices
// BN / 2 rows of each, so that a wave holds both factors of its outputs).  Stages of KS * 128 inputs
// go from memory to LDS without passing registers, NST - 1 stages ahead of the one being
// multiplied; rows and blocks past the operands' ends are given an offset past the buffer's range,
// for which the load writes zeros.
//
// Instruction st of a stage takes block KS g + st of lane group g.  A row's 16-byte blocks are
// stored so that the 16 lanes of an LDS read phase (rows 0-3, 12-15 of one lane group and rows 4-11
// of the next, or the other way round) touch 16 different 16-byte columns of the banks: see place_of.
//
// What bounds it.  8192 x 8192 x 8192 in 256 x 256 tiles: 286 us with operands out of HBM, 270 with them
// in the last-level cache, 3.8 and 4.1 PFLOP/s (a library's MXFP4 product reaches 2.9, the instruction
// alone 7.1 on random data): the matrix instructions are busy 46 % of the time, the rest is a stage's
// wait and barrier with one workgroup of 8 waves a CU.  Wider fragments a wave, loads of the next
// fragments issued earlier, two wave groups a half stage apart and a raised wave priority were measured
// and changed nothing or cost registers and time.  1024 tokens of a 256-expert, top-6 layer of 4096 x 2048,
// gate+up, 32 x 128 tiles: the weights' bytes, 2.3 GB in 455 to 465 us (5.0 TB/s); 32 tokens, down: 351 MB
// in 72 to 74 (4.8 TB/s).  8192 tokens, down, 192 pairs an expert in 256-row tiles: 461, 3.5 TB/s; a
// quarter of each tile's rows is empty, and a workgroup finds its tile and fills its stages before the
// first of only 16.
//
// Scales take the way through registers, 16 blocks (a window: four instructions) at a time,
// double-buffered.  A lane group's four bytes go side by side, so that a fragment's scales of a
// window are one linear LDS read of 256 bytes.  (Read as they come, two bytes at a row's distance
// of 32, they cost the LDS more than the codes: half of its busy cycles at 8192^3.)
constexpr int kWindowBlocks = 16;  // blocks of a row whose scales are loaded together
// Place of lane group g's block for instruction st in LDS row `row`, in 16-byte units.
template <int KS>
__device__ inline int place_of(int row, int g, int st) {
  if (KS == 2) return (g + 4 * st) ^ ((row >> 1) & 7);
  return g ^ ((0x78 >> (2 * ((row >> 2) & 3))) & 3);  // 0 2 3 1
}

// The block of a stage that lies at `place` of LDS row `row`: place_of's inverse.
template <int KS>
__device__ inline int block_at(int row, int place) {
  if (KS == 2) {
    const int q = place ^ ((row >> 1) & 7);
    return 2 * (q & 3) + (q >> 2);
  }
  return place ^ ((0x78 >> (2 * ((row >> 2) & 3))) & 3);
}

// The 16 scale bytes from byte `at` of a matrix's `size` on (size >= 16), of which the first `left`
// (at most 16, none if negative) belong to the row; the others become 127, a factor of one for the
// zero codes there.  One load of any alignment, moved back where it would pass the matrix's end; its
// bytes are moved on afterwards.  (Four loads of a dword each cost the address unit four times as
// many cache lines.)  No branches: a branch in the loop over stages lets the compiler sink the
// products of all stages behind the last one.
struct __attribute__((packed, aligned(1))) Bytes16 { uint32_t w[4]; };

__device__ inline void load_window(const uint8_t* scales, int64_t at, int64_t size, uint32_t (&s)[4]) {
  const Bytes16 v = *reinterpret_cast<const Bytes16*>(scales + min(at, size - 16));
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = v.w[i];
}

__device__ inline void trim_window(int64_t at, int64_t size, int left, uint32_t (&s)[4]) {
  const int back = (int)min(max(at - (size - 16), (int64_t)0), (int64_t)15);
  typedef unsigned __int128 u128;
  const u128 v = (((u128)s[3] << 96) | ((u128)s[2] << 64) | ((u128)s[1] << 32) | s[0]) >> (8 * back);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (uint32_t)(v >> (32 * i));
    const int in = min(max(left - 4 * i, 0), 4);  // bytes inside the row
    const uint32_t mask = (uint32_t)(((uint64_t)1 << (8 * in)) - 1);
    s[i] = (w & mask) | (0x7f7f7f7fu & ~mask);
  }
}

// Byte order of a window in LDS: dword g holds lane group g's bytes in the order of instructions.
template <int KS>
__device__ inline i32x4 window_order(const uint32_t (&s)[4]) {
  i32x4 d;
  if (KS == 2) {  // instruction 2 t + st takes byte 8 t + 2 g + st
#pragma unroll
    for (int g = 0; g < 4; ++g)
      d[g] = (int)(g & 1 ? (s[g / 2] >> 16) | (s[2 + g / 2] & 0xffff0000u) : (s[g / 2] & 0xffffu) | (s[2 + g / 2] << 16));
  } else {  // instruction t takes byte 4 t + g
    const uint32_t a = __builtin_amdgcn_perm(s[1], s[0], 0x05010400), b = __builtin_amdgcn_perm(s[3], s[2], 0x05010400);
    const uint32_t c = __builtin_amdgcn_perm(s[1], s[0], 0x07030602), e = __builtin_amdgcn_perm(s[3], s[2], 0x07030602);
    d[0] = (int)((a & 0xffffu) | (b << 16));
    d[1] = (int)((a >> 16) | (b & 0xffff0000u));
    d[2] = (int)((c & 0xffffu) | (e << 16));
    d[3] = (int)((c >> 16) | (e & 0xffff0000u));
  }
  return d;
}

template <int BM, int BN, int WM, int WN, int NST, int KS, int HALVES>
__global__ __launch_bounds__(WM * WN * 64) void tiled_kernel(MxMatmulParams p, int tiles, int row_blocks) {
  constexpr int kThreads = WM * WN * 64;
  constexpr int kRows = BM + BN;                     // rows of a stage: activations, then weights
  constexpr int kStageBlocks = 4 * KS;               // 32-value blocks of a row in a stage
  constexpr int kStageBytes = kStageBlocks * kMxBlockBytes;
  constexpr int kLoads = kRows * kStageBlocks / kThreads;  // 16-byte loads of a thread and stage
  constexpr int kScaleRows = (kRows + kThreads - 1) / kThreads;
  constexpr int kWindow = 4 / KS;                    // stages of a window
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int FH = FN / HALVES;                    // fragments of one matrix
  constexpr bool kPair = FH % 2 == 0;                // two fragments side by side: 8 outputs in a lane
  static_assert(kRows * kStageBlocks % kThreads == 0 && BM * kStageBlocks % kThreads == 0, "a load is of one operand");
  static_assert((NST == 2 || NST == 4) && FH >= 1, "");
  __shared__ __attribute__((aligned(1024))) uint8_t c0[kRows * kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t c1[kRows * kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t c2[NST > 2 ? kRows * kStageBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t c3[NST > 2 ? kRows * kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t sc[2][kRows * kWindowBlocks];

  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv / WN, wn = wv % WN;
  const int j = lane & 15, g = lane >> 4;

  int tile, rb;
  tile_of_block(p, tiles, row_blocks, (int)blockIdx.x, tile, rb);
  if (tile >= tiles) return;
  int expert = 0, start = tile * BM, len = min(BM, p.m - start);
  if (p.offsets && !find_tile(p.offsets, p.E, p.m, BM, tile, expert, start, len)) return;
  const int n0 = rb * (BN / HALVES);
  const int blocks = p.blocks;
  const size_t row_codes = (size_t)blocks * kMxBlockBytes;

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

  // Dense activations are addressed from the tile's first row, gathered ones from row 0 (a plan
  // keeps them under 2^30 bytes).
  const int a_base = p.offsets ? 0 : start;
  const size_t w_base = ((size_t)expert * p.n + n0) * row_codes;
  const __amdgpu_buffer_rsrc_t ra = product_rsrc(p.a + (size_t)a_base * row_codes);
  const __amdgpu_buffer_rsrc_t rw0 = product_rsrc(p.w0 + w_base);
  const __amdgpu_buffer_rsrc_t rw1 = product_rsrc(HALVES == 2 ? p.w1 + w_base : p.w0 + w_base);

  // Load i of a thread: LDS row and block of the stage.
  auto load_at = [&](int i, int& r, int& block) {
    const int slot = i * kThreads + tid;
    r = slot / kStageBlocks;
    block = block_at<KS>(r, slot % kStageBlocks);
  };
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    int r, block;
    load_at(i, r, block);
    if (i * kThreads < BM * kStageBlocks) {
      const int row = act_row(r);
      off[i] = row < 0 ? kNoRow : (uint32_t)((size_t)(row - a_base) * row_codes) + block * kMxBlockBytes;
    } else {
      int half;
      const int row = weight_row(r - BM, half);
      off[i] = row < p.n ? (uint32_t)((size_t)(row - n0) * row_codes) + block * kMxBlockBytes : kNoRow;
    }
  }
  const int stages = (blocks + kStageBlocks - 1) / kStageBlocks;
  auto issue = [&](uint8_t* dst, int s) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // blocks past the row's end, and stages past the last
      int r, block;
      load_at(i, r, block);
      const uint32_t o = s * kStageBlocks + block < blocks ? off[i] : kNoRow;
      const int so = min(s, stages) * kStageBytes;
      lds_void* at = (lds_void*)(dst + (i * kThreads + wv * 64) * 16);
      if (i * kThreads < BM * kStageBlocks) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, at, 16, o, so, 0, 0);
      } else {
        int half = 0;  // a wave's load is of rows of one fragment, so of one matrix
        if (HALVES == 2) weight_row((i * kThreads + wv * 64) / kStageBlocks - BM, half);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(half ? rw1 : rw0, at, 16, o, so, 0, 0);
      }
    }
  };

  // A row that is not there reads another row's scales: they reach only outputs that are not stored.
  const uint8_t* sbase[kScaleRows];
  int64_t srow[kScaleRows], ssize[kScaleRows];
#pragma unroll
  for (int i = 0; i < kScaleRows; ++i) {
    const int r = min(i * kThreads + tid, kRows - 1);
    if (r < BM) {
      sbase[i] = p.a_scale;
      srow[i] = (int64_t)max(act_row(r), 0) * blocks;
      ssize[i] = (int64_t)p.a_rows * blocks;
    } else {
      int half;
      const int row = min(weight_row(r - BM, half), p.n - 1);
      sbase[i] = half ? p.w1_scale : p.w0_scale;
      srow[i] = ((int64_t)expert * p.n + row) * blocks;
      ssize[i] = (int64_t)p.E * p.n * blocks;
    }
  }
  uint32_t sreg[kScaleRows][4];
  auto scales_load = [&](int window) {
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i)
      load_window(sbase[i], srow[i] + min(window * kWindowBlocks, blocks), ssize[i], sreg[i]);
  };
  auto scales_store = [&](int window) {
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
      const int first = min(window * kWindowBlocks, blocks);
      trim_window(srow[i] + first, ssize[i], blocks - first, sreg[i]);
      const int r = min(i * kThreads + tid, kRows - 1);  // threads past the rows write the last one's again
      *reinterpret_cast<i32x4*>(&sc[window & 1][r * kWindowBlocks]) = window_order<KS>(sreg[i]);
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int a_row = wm * (BM / WM) + j, w_row = BM + wn * (BN / WN) + j;
  int sa[FM], sw[FN];  // scales of a window
  auto read_scales = [&](int window) {
    const uint8_t* ss = &sc[window & 1][4 * g];
#pragma unroll
    for (int a = 0; a < FM; ++a) sa[a] = *reinterpret_cast<const int*>(ss + (a_row + 16 * a) * kWindowBlocks);
#pragma unroll
    for (int b = 0; b < FN; ++b) sw[b] = *reinterpret_cast<const int*>(ss + (w_row + 16 * b) * kWindowBlocks);
  };
  i32x4 fa[FM], fw[FN];
  auto read_fragments = [&](const uint8_t* cur, int st) {
    const int col = place_of<KS>(j, g, st) * 16;  // rows 16 apart have the same order of places
#pragma unroll
    for (int b = 0; b < FN; ++b) fw[b] = *reinterpret_cast<const i32x4*>(cur + (w_row + 16 * b) * kStageBytes + col);
#pragma unroll
    for (int a = 0; a < FM; ++a) fa[a] = *reinterpret_cast<const i32x4*>(cur + (a_row + 16 * a) * kStageBytes + col);
  };
  auto multiply = [&](auto byte) {  // the scales' byte of this instruction step
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
        acc[a][b] = mfma_fp4<decltype(byte)::value>(fw[b], fa[a], acc[a][b], sw[b], sa[a]);
  };

  // One stage of a window, at its place `step` there.  Before a stage is read, its codes have to have
  // arrived (the stages after it stay in flight) and every wave has to have read the stage whose
  // place the next load takes.
  auto stage = [&](const uint8_t* cur, uint8_t* next, int s, auto step_of_window) {
    constexpr int step = decltype(step_of_window)::value;
    const int window = s / kWindow;
    wait_loads<(NST - 2) * kLoads>();
    wave_barrier();
    issue(next, s + NST - 1);
    if (step == 0) {
      scales_load(window + 1);
      read_scales(window);
    }
    read_fragments(cur, 0);
    multiply(Step<KS * step>());
    if (KS == 2) {
      __builtin_amdgcn_sched_barrier(0);  // one instruction step's fragments at a time in registers
      read_fragments(cur, 1);
      multiply(Step<KS * step + KS - 1>());
    }
    if (step == kWindow - 1) scales_store(window + 1);
  };

  scales_load(0);
  issue(c0, 0);
  if (NST > 2) {
    issue(c1, 1);
    issue(c2, 2);
  }
  scales_store(0);
  // Whole turns: the stages past the last one multiply zeros.
  if (NST == 2 && KS == 2) {
    for (int s = 0; s < stages; s += 2) {
      stage(c0, c1, s, Step<0>());
      stage(c1, c0, s + 1, Step<1 % kWindow>());
    }
  } else {
    for (int s = 0; s < stages; s += 4) {
      stage(c0, NST == 2 ? c1 : c3, s, Step<0>());
      stage(c1, c0, s + 1, Step<1 % kWindow>());
      stage(NST == 2 ? c0 : c2, c1, s + 2, Step<2 % kWindow>());
      stage(NST == 2 ? c1 : c3, NST == 2 ? c0 : c2, s + 3, Step<3 % kWindow>());
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // no load to LDS outlives the workgroup

  // Lane j + 16 g of fragment (a, b): activation row 16 a + j, weight rows 4 g .. 4 g + 3 of b.
  constexpr int kSpan = kPair ? 8 : 4;
  auto write = [&](auto store) {
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      const int r = tile_row(p, start, len, wm * (BM / WM) + 16 * a + j);
#pragma unroll
      for (int b = 0; b < FH; b += kPair ? 2 : 1) {
        float v[kSpan];
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
          v[i] = acc[a][b + i / 4][i % 4];
          if (HALVES == 2) v[i] = swiglu(v[i], acc[a][(HALVES - 1) * FH + b + i / 4][i % 4]);
        }
        const int c = n0 + wn * (FH * 16) + (kPair ? 16 * b + 8 * g : 16 * b + 4 * g);
        if (r >= 0) store(r, c, v);
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

template <int BM, int BN, int WM, int WN, int NST, int KS, int HALVES>
hipError_t launch_tiled(const MxMatmulParams& p, hipStream_t stream, bool launch) {
  int64_t tiles = ((int64_t)p.m + BM - 1) / BM;
  if (p.offsets) tiles = p.m / BM + (p.m < p.E ? p.m : p.E);
  const int64_t row_blocks = ((int64_t)p.n + BN / HALVES - 1) / (BN / HALVES);
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds * row_blocks;
  if (grid * (WM * WN * 64) > kMostThreads) return hipErrorInvalidConfiguration;
  if (!launch) return hipSuccess;
  hipLaunchKernelGGL((tiled_kernel<BM, BN, WM, WN, NST, KS, HALVES>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, stream,
                     p, (int)tiles, (int)row_blocks);
  return hipGetLastError();
}

// Which kernel and tile.  Large tiles read the operands less often, small ones make more workgroups;
// below about one workgroup a CU the second counts more.  Times in us at m x n x k, or pairs of a
// 256-expert, top-6 layer of 4096 x 2048 (gate+up), each side of a border:
//   few rows             m = 1: direct; 48 x 4096 x 4096 direct 8.0, 32 x 128 9.0;
//                        48 x 8192 x 2048 direct 8.2, 32 x 128 7.2
//   256 x 256 from 256   2048 x 8192 x 2048 (256 tiles) 25.0, 128 x 128 29.6;
//     workgroups         2048 x 4096 x 4096 (128 tiles) 34.1, 128 x 128 27.2
//   128 x 128 from 200   1024 x 4096 x 4096 (256) 16.6, 64 x 128 17.6; 512 x 4096 x 4096 (128) 14.8, 11.8
//   64 x 128 from 256    512 x 4096 x 4096 (256) 11.8, 32 x 128 13.4; 256 x 4096 x 4096 (128) 10.7, 10.1
//   32 x 128: four       one workgroup a CU: nobody hides its waits.  256 x 4096 x 4096 (256) four 8.9,
//     stages up to 256   two 10.1; 300 x 2048 x 4096 (160) 8.7, 9.7; 256 x 8192 x 2048 (512) 10.7, 8.3
//   32 x 64 below 128    256 x 2048 x 4096 (128) 32 x 64 7.8, 32 x 128 8.3; 64 x 8192 x 2048 (128) 6.8, 6.3;
//     of 32 x 128        128 x 2048 x 4096 (64) 7.7, 8.2; 128 x 8192 x 2048 (256) 7.3, 6.7
//   experts              6 pairs direct 13.5, 32 x 128 15.8; 12 pairs 21.2, 20.0; 24 pairs an expert 32 x 128 458,
//                        128 x 128 485; 48 pairs 588, 533; 96 pairs 128 x 128 565, 256 x 256 659; 192 pairs 1050, 752
// The experts' points are of uniform routing, where every tile makes thousands of workgroups.  Of few or small
// experts the large tiles make fewer than there are CUs, and under skewed routing the average says little
// about a woken expert's pairs: neither is measured, and the rule does not ask.
// Without `launch` it says whether the launch could be made.
template <int HALVES>
hipError_t launch_halves(const MxMatmulParams& p, hipStream_t stream, bool launch) {
  // the tiled kernel reads 16 scales at a time and addresses a tile's rows by 31-bit offsets
  const bool tiles = (int64_t)p.a_rows * p.blocks >= 16 && (int64_t)p.E * p.n * p.blocks >= 16 && p.blocks < 1 << 18;
  if (p.offsets) {
    const int64_t row_blocks = ((int64_t)p.n + 15) / 16;
    if (p.m <= 8 || (p.m <= 16 && p.m * row_blocks <= 1280)) return launch_direct<1, HALVES, 4>(p, stream, launch);
    if (!tiles) return launch_direct<2, HALVES, 4>(p, stream, launch);
    const int fill = (p.m + p.E - 1) / p.E;  // pairs an expert gets on average
    if (fill <= 28) return launch_tiled<32, 128, 1, 4, 2, 2, HALVES>(p, stream, launch);
    if (fill <= 160) return launch_tiled<128, 128, 2, 2, 4, 1, HALVES>(p, stream, launch);
    return launch_tiled<256, 256, 2, 4, 4, 1, HALVES>(p, stream, launch);
  }
  if constexpr (HALVES == 1) {  // a dense product is of one matrix
    if (p.m <= 16 && p.blocks >= 128) return launch_direct<1, 1, 8>(p, stream, launch);
    if (p.m <= 16) return launch_direct<1, 1, 4>(p, stream, launch);
    if (!tiles || (p.m <= 64 && p.n <= 4096)) return launch_direct<2, 1, 4>(p, stream, launch);
    auto groups = [&](int64_t bm, int64_t bn) { return (p.m + bm - 1) / bm * ((p.n + bn - 1) / bn); };
    if (groups(256, 256) >= 256) return launch_tiled<256, 256, 2, 4, 4, 1, 1>(p, stream, launch);
    if (groups(128, 128) >= 200) return launch_tiled<128, 128, 2, 2, 2, 2, 1>(p, stream, launch);
    if (groups(64, 128) >= 256) return launch_tiled<64, 128, 1, 4, 2, 2, 1>(p, stream, launch);
    if (groups(32, 128) > 256) return launch_tiled<32, 128, 1, 4, 2, 2, 1>(p, stream, launch);
    if (groups(32, 128) >= 128) return launch_tiled<32, 128, 1, 4, 4, 2, 1>(p, stream, launch);
    return launch_tiled<32, 64, 1, 2, 4, 2, 1>(p, stream, launch);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulParams& p, hipStream_t stream) {
  return p.w1 ? launch_halves<2>(p, stream, true) : launch_halves<1>(p, stream, true);
}

bool mx_matmul_fits(const MxMatmulParams& p) {
  return (p.w1 ? launch_halves<2>(p, nullptr, false) : launch_halves<1>(p, nullptr, false)) == hipSuccess;
}

}  // namespace qtip
