// MXFP4 quantisation: rows of bf16, fp16 or fp32 values into blocks of 32 e2m1 codes that share
// one e8m0 scale.
//
//   floor rule:   scale = 2^(floor(log2 amax) - 2)   (2 = the exponent of the largest code, 6)
//   nearest rule: the same with amax rounded to the nearest power of two's code first: one step
//                 larger when amax >= 1.75 * 2^floor(log2 amax), so that amax / scale < 7
//   code = the e2m1 value nearest to x / scale (a tie: the even code), at most 6
//
// The scale's exponent is read from the bits of amax (no logarithm).  A block that holds a NaN or
// an infinity gets the scale 255 (NaN) and zero codes: it stands for NaN as a whole.  The last
// block of a row whose length is no multiple of 32 counts as filled up with zeros.
#include "mx_internal.h"

#include <hip/hip_bf16.h>

namespace qtip {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kPerThread = 8;  // values of one thread; four neighbouring threads hold a block

// The e2m1 code of x * inv, x finite.  inv is a power of two, in two factors because 2^(127 - byte)
// alone can leave fp32's range; the products are exact unless they fall below every border.
__device__ inline uint32_t e2m1_code(float x, float inv0, float inv1) {
  const float a = fabsf(x) * inv0 * inv1;
  uint32_t c = 0;
  c += a > 0.25f;
  c += a >= 0.75f;
  c += a > 1.25f;
  c += a >= 1.75f;
  c += a > 2.5f;
  c += a >= 3.5f;
  c += a > 5.0f;
  return c | (__builtin_bit_cast(uint32_t, x) >> 28 & 8u);
}

__device__ inline float e2m1_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float mag = m < 2 ? 0.5f * (float)m : (float)(2u + (m & 1u)) * (float)(1u << (m >> 1)) * 0.25f;
  return c & 8u ? -mag : mag;
}

__device__ inline float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

template <typename T> __device__ inline float load_one(const T* p);
template <> __device__ inline float load_one<uint16_t>(const uint16_t* p) {
  return __builtin_bit_cast(float, (uint32_t)*p << 16);
}
template <> __device__ inline float load_one<_Float16>(const _Float16* p) { return (float)*p; }
template <> __device__ inline float load_one<float>(const float* p) { return *p; }

__device__ inline void store_one(uint16_t* p, float v) {  // v is a bf16 value
  *p = (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16);
}
__device__ inline void store_one(_Float16* p, float v) { *p = (_Float16)v; }
__device__ inline void store_one(float* p, float v) { *p = v; }

template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(MxQuantParams p) {
  const int blocks = (p.cols + kMxBlock - 1) / kMxBlock;
  const int64_t per_row = (int64_t)blocks * (kMxBlock / kPerThread);
  const int64_t item = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x;
  if (item >= per_row * p.rows) return;  // a block's four threads leave together
  const int64_t row = item / per_row;
  const int part = (int)(item - row * per_row);
  const int c0 = part * kPerThread;
  const T* src = reinterpret_cast<const T*>(p.src) + row * p.row_stride;
  float v[kPerThread];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    v[i] = c0 + i < p.cols ? load_one(src + c0 + i) : 0.0f;
    top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);  // magnitudes order as integers
  }
  top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
  const bool bad = top >= 0x7f800000u;
  if (p.nearest) top += 0x200000u;
  const int field = (int)(top >> 23);
  const int byte = bad ? 255 : max(field - 2, 0);
  uint32_t packed = 0;
  const int up = (127 - byte) >> 1;
  const float inv0 = pow2(up), inv1 = pow2(127 - byte - up);
  const float s0 = pow2(-up), s1 = pow2(up - (127 - byte));
  float value[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const uint32_t c = bad ? 0u : e2m1_code(v[i], inv0, inv1);
    packed |= c << (4 * i);
    value[i] = bad ? __builtin_nanf("") : e2m1_value(c) * s0 * s1;
  }
  *reinterpret_cast<uint32_t*>(p.codes + row * blocks * kMxBlockBytes + part * 4) = packed;
  if ((part & 3) == 0) p.scales[row * blocks + (part >> 2)] = (uint8_t)byte;
  if (p.values) {
    T* dst = reinterpret_cast<T*>(p.values) + row * p.cols;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (c0 + i < p.cols) store_one(dst + c0 + i, value[i]);
  }
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantParams& p, hipStream_t stream) {
  const int64_t items = (int64_t)((p.cols + kMxBlock - 1) / kMxBlock) * (kMxBlock / kPerThread) * p.rows;
  const dim3 grid((unsigned)((items + kQuantThreads - 1) / kQuantThreads));
  if (p.source == kMxBf16)
    hipLaunchKernelGGL(quantize_kernel<uint16_t>, grid, dim3(kQuantThreads), 0, stream, p);
  else if (p.source == kMxF16)
    hipLaunchKernelGGL(quantize_kernel<_Float16>, grid, dim3(kQuantThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(quantize_kernel<float>, grid, dim3(kQuantThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace qtip
