// MXFP4 quantisation: rows of bf16, fp16 or fp32 values into blocks of 32 e2m1 codes that share
// one e8m0 scale.
//
//   floor rule:   scale = 2^(floor(log2 amax) - 2)   (2 = the exponent of the largest code, 6)
//   nearest rule: one step larger when amax >= 1.75 * 2^floor(log2 amax), so that amax / scale < 7
//   code = the e2m1 value nearest to x / scale (a tie: the even code), at most 6
//
// The scale's exponent is read from the bits of amax (no logarithm), and the gfx950 conversions with
// a scale (v_cvt_scalef32_pk_fp4_*) round two values at a time; they take the scale by the exponent
// bits of a float, so the byte 0 (2^-127) is the float of those bits.  A block that holds a NaN or an
// infinity gets the scale 255 (NaN) and zero codes: it stands for NaN as a whole.  The last block of
// a row whose length is no multiple of 32 counts as filled up with zeros.
//
// One pass over the values, bound by memory: eight values a thread (16 or 32 bytes, the widest loads),
// so that a block's four threads find its largest value by two lane moves without LDS, and every thread
// stores one dword of codes.  8192 x 8136 fp32 values with the values of the codes written back, 569 MB:
// 118 us, 4.8 TB/s (the copy rate; 73 to 99 vector instructions a wave of 512 values).  8192 x 8192 bf16
// to codes alone, 170 MB: 32 to 38 us.  32 x 4096: 2.4 us, the launch.  Rounding by comparisons against
// the code's borders instead of the scaled conversions took 252 us for the first.
#include "mx_internal.h"

namespace qtip {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kPerThread = 8;  // values of one thread; four neighbouring threads hold a block

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// What differs between the source types: eight values as dwords, their largest magnitude as the bits
// of a float (magnitudes order as integers), and the conversions.
struct Bf16 {
  typedef uint16_t Elem;
  static constexpr int kWords = 4;
  static __device__ uint32_t top(const uint32_t (&w)[4]) {
    u16x2 m = __builtin_bit_cast(u16x2, w[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    return (uint32_t)max(m[0], m[1]) << 16;
  }
  template <int I> static __device__ uint32_t code(uint32_t old, const uint32_t (&w)[4], float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, w[I]), scale, I);
  }
  template <int I> static __device__ void value(uint32_t codes, float scale, uint32_t (&w)[4]) {
    w[I] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
  }
  static constexpr uint32_t kNan = 0x7fc07fc0u;
};

struct F16 {
  typedef uint16_t Elem;
  static constexpr int kWords = 4;
  static __device__ uint32_t top(const uint32_t (&w)[4]) {
    const uint32_t m = Bf16::top(w) >> 16;  // the same integer order
    return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)m));
  }
  template <int I> static __device__ uint32_t code(uint32_t old, const uint32_t (&w)[4], float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, w[I]), scale, I);
  }
  template <int I> static __device__ void value(uint32_t codes, float scale, uint32_t (&w)[4]) {
    w[I] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, I));
  }
  static constexpr uint32_t kNan = 0x7e007e00u;
};

struct F32 {
  typedef uint32_t Elem;
  static constexpr int kWords = 8;
  static __device__ uint32_t top(const uint32_t (&w)[8]) {
    uint32_t m = w[0] & 0x7fffffffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
  }
  template <int I> static __device__ uint32_t code(uint32_t old, const uint32_t (&w)[8], float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __builtin_bit_cast(float, w[2 * I]),
                                                    __builtin_bit_cast(float, w[2 * I + 1]), scale, I);
  }
  template <int I> static __device__ void value(uint32_t codes, float scale, uint32_t (&w)[8]) {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, I);
    const float lo = v[0], hi = v[1];  // a bit cast of a vector's element itself reads element 0
    w[2 * I] = __builtin_bit_cast(uint32_t, lo);
    w[2 * I + 1] = __builtin_bit_cast(uint32_t, hi);
  }
  static constexpr uint32_t kNan = 0x7fc00000u;
};

template <class T, bool VALUES>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(MxQuantParams p) {
  typedef typename T::Elem Elem;
  constexpr int kWords = T::kWords;
  struct __attribute__((packed, aligned(sizeof(Elem)))) Eight { uint32_t w[kWords]; };  // at any element's address
  const uint32_t blocks = ((uint32_t)p.cols + kMxBlock - 1) / kMxBlock;
  const int64_t item = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x;
  const uint32_t block = (uint32_t)(item >> 2);  // rows x blocks < 2^30
  if (block >= blocks * (uint32_t)p.rows) return;  // a block's four threads leave together
  const uint32_t row = block / blocks;
  const int part = (int)((block - row * blocks) * 4) + (int)(item & 3);
  const int c0 = part * kPerThread;  // at most 2^31 - 8
  const int left = p.cols - c0;      // of the row, these eight and what follows; below 0 past its end
  const Elem* src = reinterpret_cast<const Elem*>(p.src) + (int64_t)row * p.row_stride + c0;
  uint32_t w[kWords];
  if (left >= kPerThread) {
    const Eight v = *reinterpret_cast<const Eight*>(src);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = v.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (i < left) w[i * kWords / 8] |= (uint32_t)src[i] << (kWords == 4 ? 16 * (i & 1) : 0);
  }
  uint32_t top = T::top(w);
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));  // quad lanes 1 0 3 2
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));  // quad lanes 2 3 0 1
  const bool bad = top >= 0x7f800000u;
  if (p.nearest) top += 0x200000u;
  const uint32_t byte = bad ? 255u : (uint32_t)max((int)(top >> 23) - 2, 0);
  const float scale = __builtin_bit_cast(float, byte << 23);
  uint32_t codes = 0;
  codes = T::template code<0>(codes, w, scale);
  codes = T::template code<1>(codes, w, scale);
  codes = T::template code<2>(codes, w, scale);
  codes = T::template code<3>(codes, w, scale);
  if (bad) codes = 0;
  *reinterpret_cast<uint32_t*>(p.codes + (size_t)block * kMxBlockBytes + (item & 3) * 4) = codes;
  if ((item & 3) == 0) p.scales[block] = (uint8_t)byte;
  if (VALUES) {
    Elem* dst = reinterpret_cast<Elem*>(p.values) + (int64_t)row * p.cols + c0;
    Eight v;
    T::template value<0>(codes, scale, v.w);
    T::template value<1>(codes, scale, v.w);
    T::template value<2>(codes, scale, v.w);
    T::template value<3>(codes, scale, v.w);
    if (bad) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) v.w[i] = T::kNan;
    }
    if (left >= kPerThread) {
      *reinterpret_cast<Eight*>(dst) = v;
    } else {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (i < left) dst[i] = (Elem)(v.w[i * kWords / 8] >> (kWords == 4 ? 16 * (i & 1) : 0));
    }
  }
}

template <class T>
void launch_source(const MxQuantParams& p, dim3 grid, hipStream_t stream) {
  if (p.values)
    hipLaunchKernelGGL((quantize_kernel<T, true>), grid, dim3(kQuantThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((quantize_kernel<T, false>), grid, dim3(kQuantThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantParams& p, hipStream_t stream) {
  const int64_t items = ((int64_t)p.cols + kMxBlock - 1) / kMxBlock * (kMxBlock / kPerThread) * p.rows;
  const dim3 grid((unsigned)((items + kQuantThreads - 1) / kQuantThreads));
  if (p.source == kMxBf16) launch_source<Bf16>(p, grid, stream);
  else if (p.source == kMxF16) launch_source<F16>(p, grid, stream);
  else launch_source<F32>(p, grid, stream);
  return hipGetLastError();
}

}  // namespace qtip
