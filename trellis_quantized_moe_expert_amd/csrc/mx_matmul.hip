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

__device__ inline uint32_t bf16_bits(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;  // NaN stays one
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

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
    const int c0 = n0 + 4 * (ln >> 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c0 + i >= p.n) break;
      float v = y[0][i];
      if (HALVES == 2) v = v / (1.0f + expf(-v)) * y[HALVES - 1][i];
      const size_t o = (size_t)r * p.n + c0 + i;
      if (p.out_bf16) reinterpret_cast<uint16_t*>(p.out)[o] = (uint16_t)bf16_bits(v);
      else reinterpret_cast<float*>(p.out)[o] = v;
    }
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

}  // namespace

hipError_t launch_mx_matmul(const MxMatmulParams& p, hipStream_t stream) {
  return p.m <= 16 ? launch_direct<1>(p, stream) : launch_direct<4>(p, stream);
}

}  // namespace qtip
