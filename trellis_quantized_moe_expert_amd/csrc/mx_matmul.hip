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
#include "qtip_internal.h"

#include <cmath>

namespace qtip {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the operand format of the f8f6f4 instructions: e2m1

template <int SEL>
__device__ inline f32x4 mfma_fp4(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  const i32x8 a8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8{b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, kFp4, kFp4, SEL, sa, SEL, sb);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ inline uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// silu(g) u.  exp(-g) = inf makes the reciprocal 0 and the result -0, the limit.
__device__ inline float swiglu(float g, float u) { return g * __builtin_amdgcn_rcpf(1.0f + expf(-g)) * u; }

// The t-th tile of at most bm pairs of one expert, experts ascending: its expert, first place in
// sorted_pair and number of pairs.  One wave finds it from the bins' offsets; false past the last.
__device__ inline bool find_tile(const int32_t* __restrict__ offsets, int E, int pairs, int bm, int t, int& expert,
                                 int& start, int& len) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;  // consecutive experts of one lane
  const int e0 = lane * per;
  auto count = [&](int e, int& lo) {
    lo = min(max(offsets[e], 0), pairs);
    return max(min(max(offsets[e + 1], 0), pairs) - lo, 0);
  };
  int tiles = 0;
  for (int i = 0; i < per; ++i)
    if (e0 + i < E) {
      int lo;
      tiles += (count(e0 + i, lo) + bm - 1) / bm;
    }
  int incl = tiles;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(incl, off, 64);
    if (lane >= off) incl += up;
  }
  const uint64_t past = __ballot(incl > t);
  if (past == 0) return false;
  const int owner = __ffsll((unsigned long long)past) - 1;
  int rest = t - (incl - tiles), ex = 0, st = 0, ln = 0;
  if (lane == owner) {
    for (int i = 0; i < per; ++i) {
      int lo;
      const int c = count(e0 + i, lo), nt = (c + bm - 1) / bm;
      if (rest < nt) {
        ex = e0 + i;
        st = lo + rest * bm;
        ln = min(bm, c - rest * bm);
        break;
      }
      rest -= nt;
    }
  }
  expert = __builtin_amdgcn_readlane(ex, owner);
  start = __builtin_amdgcn_readlane(st, owner);
  len = __builtin_amdgcn_readlane(ln, owner);
  return true;
}

// Rows of the output tile: the pair ids (or dense rows) of a tile; -1 where there is none.
__device__ inline int tile_row(const MxMatmulParams& p, int start, int len, int i) {
  if (i >= len) return -1;
  if (!p.offsets) return start + i;
  const int r = p.sorted_pair[start + i];
  return r >= 0 && r < p.m ? r : -1;
}

// Stores SPAN neighbouring outputs of row r from column c on: a whole vector where p.n is a multiple
// of SPAN (so that it lies in the row or past it, aligned), one by one otherwise.
template <int SPAN>
__device__ inline void store_bf16(const MxMatmulParams& p, int r, int c, const float (&v)[SPAN]) {
  if (c >= p.n) return;
  uint32_t w[SPAN / 2];
#pragma unroll
  for (int i = 0; i < SPAN / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  __bf16* d = reinterpret_cast<__bf16*>(p.out) + (size_t)r * p.n + c;
  if (SPAN == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[SPAN / 2 - 2], w[SPAN / 2 - 1]);
  else *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
}

template <int SPAN>
__device__ inline void store_f32(const MxMatmulParams& p, int r, int c, const float (&v)[SPAN]) {
  if (c >= p.n) return;
  float* d = reinterpret_cast<float*>(p.out) + (size_t)r * p.n + c;
#pragma unroll
  for (int i = 0; i < SPAN; i += 4) *reinterpret_cast<float4*>(d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

template <int SPAN>
__device__ inline void store_odd(const MxMatmulParams& p, int r, int c, const float (&v)[SPAN]) {
  const size_t o = (size_t)r * p.n + c;
#pragma unroll
  for (int i = 0; i < SPAN; ++i) {
    if (c + i >= p.n) break;
    if (p.out_bf16) reinterpret_cast<__bf16*>(p.out)[o + i] = (__bf16)v[i];
    else reinterpret_cast<float*>(p.out)[o + i] = v[i];
  }
}

constexpr int kXcds = 8;  // workgroups go round-robin over the XCDs of an MI355X, each with its own L2

// The tile (of activation rows) and row block (of weight rows) of a workgroup.  Expert tiles go to
// the XCDs in turn, a tile's row blocks all to one: its activations stay in that XCD's L2, and the
// tiles past the last one (the grid is sized for the most there can be) are spread evenly.  Dense
// products give each XCD a run of consecutive blocks, walked down columns of 8 tiles, so that the
// blocks running at a time share few operand rows.
__device__ inline void tile_of_block(const MxMatmulParams& p, int tiles, int row_blocks, int b, int& tile, int& rb) {
  const int xcd = b % kXcds, i = b / kXcds;
  if (p.offsets) {
    tile = i / row_blocks * kXcds + xcd;
    rb = i % row_blocks;
    return;
  }
  const int padded = (tiles + kXcds - 1) / kXcds * kXcds;
  const int at = xcd * (padded / kXcds * row_blocks) + i;  // a bijection: the grid is padded * row_blocks
  const int column = at / (8 * row_blocks), in = at % (8 * row_blocks);
  tile = column * 8 + in % 8;
  rb = in / 8;
}

constexpr int kDirectWaves = 8;

// One workgroup: 16 weight rows (of both matrices where there are two) by MB * 16 activation rows;
// its waves split the inputs, run by run of 512, and add their sums through LDS.
template <int MB, int HALVES>
__global__ __launch_bounds__(kDirectWaves * 64) void direct_kernel(MxMatmulParams p) {
  __shared__ f32x4 red[kDirectWaves][HALVES * MB][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
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

  auto load = [&](const uint8_t* codes, const uint8_t* scales, int first, i32x4 (&c)[4], int& s) {
    s = 0;
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      c[st] = i32x4{0, 0, 0, 0};
      if (first + st < p.blocks) {
        c[st] = *reinterpret_cast<const i32x4*>(codes + (size_t)(first + st) * kMxBlockBytes);
        s |= (int)scales[first + st] << (8 * st);
      } else {
        s |= 127 << (8 * st);
      }
    }
  };
  for (int run = wv; run * 16 < p.blocks; run += kDirectWaves) {
    const int first = run * 16 + 4 * g;
    i32x4 w[HALVES][4], a[MB][4];
    int sw[HALVES], sa[MB];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) load(wc[h], ws[h], first, w[h], sw[h]);
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
  }
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int b = 0; b < MB; ++b) red[wv][h * MB + b][lane] = acc[h][b];
  __syncthreads();
  // Lane j + 16 g of fragment b holds weight rows n0 + 4g .. + 3 of activation row 16 b + j.
  for (int q = threadIdx.x; q < MB * 64; q += kDirectWaves * 64) {
    const int b = q >> 6, ln = q & 63;
    const int r = tile_row(p, start, len, 16 * b + (ln & 15));
    if (r < 0) continue;
    f32x4 y[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      y[h] = red[0][h * MB + b][ln];
      for (int u = 1; u < kDirectWaves; ++u) y[h] += red[u][h * MB + b][ln];
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

template <int MB>
hipError_t launch_direct(const MxMatmulParams& p, hipStream_t stream) {
  int64_t tiles = (p.m + MB * 16 - 1) / (MB * 16);
  // an expert's last tile may be partly filled: at most one more per expert that has pairs
  if (p.offsets) tiles = p.m / (MB * 16) + (p.m < p.E ? p.m : p.E);
  const int64_t grid = tiles * ((p.n + 15) / 16);
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  if (p.w1)
    hipLaunchKernelGGL((direct_kernel<MB, 2>), dim3((unsigned)grid), dim3(kDirectWaves * 64), 0, stream, p);
  else
    hipLaunchKernelGGL((direct_kernel<MB, 1>), dim3((unsigned)grid), dim3(kDirectWaves * 64), 0, stream, p);
  return hipGetLastError();
}


// ---- the tiled kernel -----------------------------------------------------------------------
// A workgroup of WM x WN waves computes BM activation rows by BN weight rows (with two matrices
// BN / 2 rows of each, so that a wave holds both factors of its outputs).  Stages of 256 inputs
// (128 bytes a row) go from memory to LDS without passing registers, NST - 1 stages ahead of the
// one being multiplied; rows and blocks past the operands' ends are given an offset past the
// buffer's range, for which the load writes zeros.
//
// The 16-byte blocks of a row are stored so that the 16 lanes of an LDS read phase touch 16
// different 16-byte columns: the block 2g + st of a stage (lane group g, instruction st) lies at
// place (g + 4 st) ^ ((row / 2) % 8).
//
// Scales take the way through registers, four stages (32 bytes a row) at a time, double-buffered.
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kStageBlocks = 8;           // 32-value blocks of a row in a stage
constexpr int kStageBytes = 128;          // their codes
constexpr int kWindow = 4;                // stages whose scales are loaded together
constexpr int kWindowBytes = kWindow * kStageBlocks;
constexpr uint32_t kNoRow = 0x80000000u;  // a byte offset past every buffer resource's range

__device__ inline __amdgpu_buffer_rsrc_t mx_rsrc(const uint8_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, 0x7fffffff, 0x00020000);
}

// The 32 scale bytes of one row's window from block `first` on; 127 (a factor of one, for the zero
// codes) past the row's end.  Rows of scales need no alignment: the loads are dwords of any address,
// those at the row's end moved back to end with it (blocks >= 4).  No branches: a branch in the loop
// over stages lets the compiler sink the products of all stages behind the last one.
__device__ inline void load_window(const uint8_t* row, int first, int blocks, uint32_t (&s)[8]) {
  typedef uint32_t __attribute__((aligned(1))) u32_any;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = first + 4 * i;
    s[i] = *reinterpret_cast<const u32_any*>(row + min(at, blocks - 4));
  }
}

__device__ inline void trim_window(int first, int blocks, uint32_t (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int left = min(max(blocks - (first + 4 * i), 0), 4);  // bytes inside the row
    const uint32_t v = (uint32_t)(((uint64_t)s[i]) >> (8 * (4 - left)));
    const uint32_t mask = (uint32_t)(((uint64_t)1 << (8 * left)) - 1);
    s[i] = (v & mask) | (0x7f7f7f7fu & ~mask);
  }
}

template <int BM, int BN, int WM, int WN, int NST, int HALVES>
__global__ __launch_bounds__(WM * WN * 64) void tiled_kernel(MxMatmulParams p, int tiles, int row_blocks) {
  constexpr int kThreads = WM * WN * 64;
  constexpr int kRows = BM + BN;                     // rows of a stage: activations, then weights
  constexpr int kLoads = kRows * 8 / kThreads;       // 16-byte loads of a thread and stage
  constexpr int kScaleRows = (kRows + kThreads - 1) / kThreads;
  constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr int FH = FN / HALVES;                    // fragments of one matrix
  constexpr bool kPair = FH % 2 == 0;                // two fragments side by side: 8 outputs in a lane
  static_assert(kRows * 8 % kThreads == 0 && (NST == 2 || NST == 4), "");
  __shared__ __attribute__((aligned(1024))) uint8_t c0[kRows * kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t c1[kRows * kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t c2[NST > 2 ? kRows * kStageBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t c3[NST > 2 ? kRows * kStageBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t sc[2][kRows * kWindowBytes];

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
  const __amdgpu_buffer_rsrc_t ra = mx_rsrc(p.a + (size_t)a_base * row_codes);
  const __amdgpu_buffer_rsrc_t rw0 = mx_rsrc(p.w0 + w_base);
  const __amdgpu_buffer_rsrc_t rw1 = mx_rsrc(HALVES == 2 ? p.w1 + w_base : p.w0 + w_base);

  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int slot = i * kThreads + tid, r = slot >> 3;
    const int place = (slot & 7) ^ ((r >> 1) & 7);
    const int block = 2 * (place & 3) + (place >> 2);
    if (i * kThreads < BM * 8) {
      const int row = act_row(r);
      off[i] = row < 0 ? kNoRow : (uint32_t)((size_t)(row - a_base) * row_codes) + block * kMxBlockBytes;
    } else {
      int half;
      const int row = weight_row(r - BM, half);
      off[i] = row < p.n ? (uint32_t)((size_t)(row - n0) * row_codes) + block * kMxBlockBytes : kNoRow;
    }
  }
  static_assert(BM * 8 % kThreads == 0, "a load index is of one operand");
  const int stages = (blocks + kStageBlocks - 1) / kStageBlocks;
  auto issue = [&](uint8_t* dst, int s) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // blocks past the row's end, and stages past the last
      const int slot = i * kThreads + tid, place = (slot & 7) ^ ((slot >> 4) & 7);
      const uint32_t o = s * kStageBlocks + 2 * (place & 3) + (place >> 2) < blocks ? off[i] : kNoRow;
      const int so = min(s, stages) * kStageBytes;
      lds_void* at = (lds_void*)(dst + (i * kThreads + wv * 64) * 16);
      if (i * kThreads < BM * 8) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, at, 16, o, so, 0, 0);
      } else {
        int half = 0;  // a wave's load is of 8 rows of one fragment, so of one matrix
        if (HALVES == 2) weight_row((i * kThreads + wv * 64) / 8 - BM, half);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(half ? rw1 : rw0, at, 16, o, so, 0, 0);
      }
    }
  };

  // A row that is not there reads another row's scales: they reach only outputs that are not stored.
  const uint8_t* srow[kScaleRows];
#pragma unroll
  for (int i = 0; i < kScaleRows; ++i) {
    const int r = min(i * kThreads + tid, kRows - 1);
    if (r < BM) {
      srow[i] = p.a_scale + (size_t)max(act_row(r), 0) * blocks;
    } else {
      int half;
      const int row = min(weight_row(r - BM, half), p.n - 1);
      srow[i] = (half ? p.w1_scale : p.w0_scale) + ((size_t)expert * p.n + row) * blocks;
    }
  }
  uint32_t sreg[kScaleRows][8];
  auto scales_load = [&](int window) {
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) load_window(srow[i], window * kWindowBytes, blocks, sreg[i]);
  };
  auto scales_store = [&](int window) {
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
      trim_window(window * kWindowBytes, blocks, sreg[i]);
      const int r = min(i * kThreads + tid, kRows - 1);  // threads past the rows write the last one's again
      {
        i32x4* d = reinterpret_cast<i32x4*>(&sc[window & 1][r * kWindowBytes]);
        d[0] = i32x4{(int)sreg[i][0], (int)sreg[i][1], (int)sreg[i][2], (int)sreg[i][3]};
        d[1] = i32x4{(int)sreg[i][4], (int)sreg[i][5], (int)sreg[i][6], (int)sreg[i][7]};
      }
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int key = (j >> 1) & 7;
  const int a_row = wm * (BM / WM) + j, w_row = BM + wn * (BN / WN) + j;
  auto multiply = [&](const uint8_t* cur, int window, int step) {
    const uint8_t* ss = &sc[window & 1][step * kStageBlocks + 2 * g];
    int sa[FM], sw[FN];
#pragma unroll
    for (int a = 0; a < FM; ++a) sa[a] = *reinterpret_cast<const uint16_t*>(ss + (a_row + 16 * a) * kWindowBytes);
#pragma unroll
    for (int b = 0; b < FN; ++b) sw[b] = *reinterpret_cast<const uint16_t*>(ss + (w_row + 16 * b) * kWindowBytes);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      __builtin_amdgcn_sched_barrier(0);  // one instruction step's fragments at a time in registers
      const int col = ((g + 4 * st) ^ key) * 16;
      i32x4 fa[FM], fw[FN];
#pragma unroll
      for (int a = 0; a < FM; ++a) fa[a] = *reinterpret_cast<const i32x4*>(cur + (a_row + 16 * a) * kStageBytes + col);
#pragma unroll
      for (int b = 0; b < FN; ++b) fw[b] = *reinterpret_cast<const i32x4*>(cur + (w_row + 16 * b) * kStageBytes + col);
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = st == 0 ? mfma_fp4<0>(fw[b], fa[a], acc[a][b], sw[b], sa[a])
                              : mfma_fp4<1>(fw[b], fa[a], acc[a][b], sw[b], sa[a]);
    }
  };
  // One stage: wait for its codes (the stages after it stay in flight) and for every wave to have
  // read the stage whose place the next load takes, start that load, multiply.
  auto stage = [&](const uint8_t* cur, uint8_t* next, int s0, int step) {  // stage s0 + step, s0 % 4 == 0
    const int s = s0 + step;
    constexpr int kFly = (NST - 2) * kLoads;
    static_assert(kFly < 64, "");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kFly & 15) | (kFly >> 4) << 14 | 7 << 4);  // vmcnt(kFly) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    issue(next, s + NST - 1);
    if (step == 0) scales_load(s0 / kWindow + 1);
    multiply(cur, s0 / kWindow, step);
    if (step == kWindow - 1) scales_store(s0 / kWindow + 1);
  };

  scales_load(0);
  issue(c0, 0);
  if (NST > 2) {
    issue(c1, 1);
    issue(c2, 2);
  }
  scales_store(0);
  // Whole windows: up to three stages past the last one multiply zeros.
  for (int s = 0; s < stages; s += kWindow) {
    if (NST == 2) {
      stage(c0, c1, s, 0);
      stage(c1, c0, s, 1);
      stage(c0, c1, s, 2);
      stage(c1, c0, s, 3);
    } else {
      stage(c0, c3, s, 0);
      stage(c1, c0, s, 1);
      stage(c2, c1, s, 2);
      stage(c3, c2, s, 3);
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

template <int BM, int BN, int WM, int WN, int NST, int HALVES>
hipError_t launch_tiled(const MxMatmulParams& p, hipStream_t stream) {
  int64_t tiles = (p.m + BM - 1) / BM;
  if (p.offsets) tiles = p.m / BM + (p.m < p.E ? p.m : p.E);
  const int64_t row_blocks = (p.n + BN / HALVES - 1) / (BN / HALVES);
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds * row_blocks;
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((tiled_kernel<BM, BN, WM, WN, NST, HALVES>), dim3((unsigned)grid), dim3(WM * WN * 64), 0, stream,
                     p, (int)tiles, (int)row_blocks);
  return hipGetLastError();
}

template <int HALVES>
hipError_t launch_halves(const MxMatmulParams& p, hipStream_t stream) {
  // rows of a full tile: pairs an expert gets on average, or all rows
  const int fill = p.offsets ? (p.m + p.E - 1) / p.E : p.m;
  if (p.m <= 16) return launch_direct<1>(p, stream);
  // the tiled kernel reads scales by dwords and addresses a tile's rows by 31-bit offsets
  if (p.blocks < 4 || p.blocks >= 1 << 18) return launch_direct<4>(p, stream);
  if (fill <= 64) return launch_tiled<64, 128, 1, 4, 4, HALVES>(p, stream);
  return launch_tiled<256, 256, 2, 4, 2, HALVES>(p, stream);
}

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulParams& p, hipStream_t stream) {
  return p.w1 ? launch_halves<2>(p, stream) : launch_halves<1>(p, stream);
}

}  // namespace qtip
