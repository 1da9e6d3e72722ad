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
#include "f8_device.h"
#include "f8_internal.h"
#include "product_device.h"

namespace qtip {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A lane's 32 values of a block, widened.
struct Wide {
  bf16x8 v[4];
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
// One workgroup: 16 weight rows by MB * 16 activation rows; its W waves split the inputs, run by run of U blocks, and
// add their sums through LDS.  Operands go from memory to registers: with few activation rows a call is a
// stream of weights, and the more of them are asked for at once the better.
// TAIL: the rows do not end with a run.
template <int MB, int W, bool TAIL>
__global__ __launch_bounds__(W * 64) void direct_kernel(F8MatmulParams p) {
  constexpr int U = 4;
  __shared__ f32x4 red[W][MB][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int j = lane & 15, g = lane >> 4;
  const int row_blocks = (p.n + 15) >> 4;
  const int tile = (int)blockIdx.x / row_blocks;
  const int n0 = ((int)blockIdx.x - tile * row_blocks) * 16;
  int expert = 0, start = tile * MB * 16, len = min(MB * 16, p.m - start);
  if (p.offsets && !find_tile(p.offsets, p.E, p.m, MB * 16, tile, expert, start, len)) return;

  const int blocks = (p.k + kF8Block - 1) / kF8Block;
  int first = wv * U;
  int at = first * kF8Block + g * 16;  // this lane's first byte of the run
  const uint8_t* wc = p.w0 + ((size_t)expert * p.n + min(n0 + j, p.n - 1)) * p.k;
  const float* ws = p.w0_scale + ((size_t)expert * ((p.n + kF8Block - 1) / kF8Block) + n0 / kF8Block) * blocks;
  i32x4 w[U][2] = {};
  if (first < blocks) load_blocks<U, TAIL>(wc + at, p.k - at, w);  // before the activation rows are looked up

  const uint8_t* ac[MB];
  const float* as[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int r = tile_row(p, start, len, 16 * b + j);
    const size_t arow = (size_t)(r < 0 ? 0 : r / p.a_div);  // rows past the tile read row 0; never stored
    ac[b] = p.a + arow * p.k;
    as[b] = p.a_scale + arow * blocks;
  }
  f32x4 acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (; first < blocks; first += W * U) {
    i32x4 a[MB][U][2];
    float sw[U], sa[MB][U];
    load_scales<U, TAIL>(ws, first, blocks, sw);
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      load_blocks<U, TAIL>(ac[b] + at, p.k - at, a[b]);
      load_scales<U, TAIL>(as[b], first, blocks, sa[b]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Wide ww(w[u]);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const f32x4 part = multiply_block(ww, Wide(a[b][u]));
        const float s = sw[u] * sa[b][u];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = fmaf(part[i], s, acc[b][i]);
      }
    }
    at += W * U * kF8Block;
    if (first + W * U < blocks) load_blocks<U, TAIL>(wc + at, p.k - at, w);
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) red[wv][b][lane] = acc[b];
  __syncthreads();
  for (int q = threadIdx.x; q < MB * 64; q += W * 64) {
    const int b = q >> 6, ln = q & 63;
    const int r = tile_row(p, start, len, 16 * b + (ln & 15));
    if (r < 0) continue;
    f32x4 y = red[0][b][ln];
#pragma unroll
    for (int u = 1; u < W; ++u) y += red[u][b][ln];
    const float v[4] = {y[0], y[1], y[2], y[3]};
    const int c = n0 + 4 * (ln >> 4);
    if (p.n % 4 != 0) store_odd<4>(p, r, c, v);
    else if (p.out_bf16) store_bf16<4>(p, r, c, v);
    else store_f32<4>(p, r, c, v);
  }
}

// ---- the direct kernel of two matrices -------------------------------------------------------
// One workgroup: 128 rows of both matrices by MB * 16 activation rows, so that it holds whole blocks of its outputs and
// can leave them in 8 bits.  Wave i takes 16 rows (i % 8) of both and part i / 8 of the inputs.
template <int MB, int S>
__global__ __launch_bounds__(S * 512) void direct_pair_kernel(F8MatmulParams p) {
  constexpr int U = 2;
  __shared__ f32x4 red[S][8][2 * MB][64];
  __shared__ uint32_t tops[MB * 16][8];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int j = lane & 15, g = lane >> 4;
  const int part = wv >> 3, group = wv & 7;
  const int row_blocks = p.n / kF8Block;  // an expert's rows are whole blocks
  const int tile = (int)blockIdx.x / row_blocks, rb = (int)blockIdx.x - tile * row_blocks;
  const int n0 = rb * kF8Block + group * 16;
  int expert, start, len;
  if (!find_tile(p.offsets, p.E, p.m, MB * 16, tile, expert, start, len)) return;

  const int blocks = p.k / kF8Block;
  int first = part * U;
  int at = first * kF8Block + g * 16;
  const size_t wrow = ((size_t)expert * p.n + n0 + j) * p.k;
  const uint8_t* wc[2] = {p.w0 + wrow, p.w1 + wrow};
  const size_t wsrow = ((size_t)expert * row_blocks + rb) * blocks;
  const float* ws[2] = {p.w0_scale + wsrow, p.w1_scale + wsrow};
  i32x4 w[2][U][2] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (first < blocks) load_blocks<U, true>(wc[h] + at, p.k - at, w[h]);

  const uint8_t* ac[MB];
  const float* as[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int r = tile_row(p, start, len, 16 * b + j);
    const size_t arow = (size_t)(r < 0 ? 0 : r / p.a_div);  // rows past the tile read row 0; never stored
    ac[b] = p.a + arow * p.k;
    as[b] = p.a_scale + arow * blocks;
  }
  f32x4 acc[2][MB];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[h][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (; first < blocks; first += S * U) {
    i32x4 a[MB][U][2];
    float sw[2][U], sa[MB][U];
#pragma unroll
    for (int h = 0; h < 2; ++h) load_scales<U, true>(ws[h], first, blocks, sw[h]);
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      load_blocks<U, true>(ac[b] + at, p.k - at, a[b]);
      load_scales<U, true>(as[b], first, blocks, sa[b]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Wide ww[2] = {Wide(w[0][u]), Wide(w[1][u])};
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const Wide aa(a[b][u]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 sum = multiply_block(ww[h], aa);
          const float s = sw[h][u] * sa[b][u];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[h][b][i] = fmaf(sum[i], s, acc[h][b][i]);
        }
      }
    }
    at += S * U * kF8Block;
    if (first + S * U < blocks) {
#pragma unroll
      for (int h = 0; h < 2; ++h) load_blocks<U, true>(wc[h] + at, p.k - at, w[h]);
    }
  }
  if (part > 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < MB; ++b) red[part][group][h * MB + b][lane] = acc[h][b];
  }
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int u = 1; u < S; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[h][b] += red[u][group][h * MB + b][lane];
  }
  float v[MB][4];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[b][i] = swiglu(acc[0][b][i], acc[1][b][i]);
  if (p.out_scale) {
    if (part == 0) {
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, f8_bits(v[b][i]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        if (g == 0) tops[16 * b + j][group] = top;
      }
    }
    __syncthreads();
  }
  if (part != 0) return;
  const int c = n0 + 4 * g;
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int r = tile_row(p, start, len, 16 * b + j);
    if (r < 0) continue;
    if (p.out_scale) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, tops[16 * b + j][i]);
      const F8Scale s(top, false);
      uint32_t codes[1];
      f8_codes(v[b], s, codes);
      *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(p.out) + (size_t)r * p.n + c) = codes[0];
      if (group == 0 && g == 0) p.out_scale[(size_t)r * row_blocks + rb] = s.scale;
    } else if (p.out_bf16) {
      store_bf16<4>(p, r, c, v[b]);
    } else {
      store_f32<4>(p, r, c, v[b]);
    }
  }
}

// Tiles of at most bm rows there can be: an expert's last tile may be partly filled, at most one more per expert
// that has pairs.  64 bits: m and n go up to 2^31 - 1.
int64_t most_tiles(const F8MatmulParams& p, int bm) {
  if (p.offsets) return p.m / bm + (p.m < p.E ? p.m : p.E);
  return ((int64_t)p.m + bm - 1) / bm;
}

template <int MB, int W>
hipError_t launch_direct(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  const int64_t grid = most_tiles(p, MB * 16) * (((int64_t)p.n + 15) / 16);
  if (grid * (W * 64) > kMostThreads) return hipErrorInvalidConfiguration;
  if (!launch) return hipSuccess;
  if (p.k % (4 * kF8Block) == 0)
    hipLaunchKernelGGL((direct_kernel<MB, W, false>), dim3((unsigned)grid), dim3(W * 64), 0, stream, p);
  else
    hipLaunchKernelGGL((direct_kernel<MB, W, true>), dim3((unsigned)grid), dim3(W * 64), 0, stream, p);
  return hipGetLastError();
}

template <int MB, int S>
hipError_t launch_direct_pair(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  const int64_t grid = most_tiles(p, MB * 16) * (p.n / kF8Block);
  if (grid * (S * 512) > kMostThreads) return hipErrorInvalidConfiguration;
  if (!launch) return hipSuccess;
  hipLaunchKernelGGL((direct_pair_kernel<MB, S>), dim3((unsigned)grid), dim3(S * 512), 0, stream, p);
  return hipGetLastError();
}

// Without `launch` it says whether the launch could be made.
hipError_t choose(const F8MatmulParams& p, hipStream_t stream, bool launch) {
  if (p.w1) return p.m <= 64 ? launch_direct_pair<1, 2>(p, stream, launch) : launch_direct_pair<2, 1>(p, stream, launch);
  if (p.m <= 16) return launch_direct<1, 8>(p, stream, launch);
  return launch_direct<2, 4>(p, stream, launch);
}

}  // namespace

hipError_t launch_f8_matmul(const F8MatmulParams& p, hipStream_t stream) { return choose(p, stream, true); }

bool f8_matmul_fits(const F8MatmulParams& p) { return choose(p, nullptr, false) == hipSuccess; }

}  // namespace qtip
