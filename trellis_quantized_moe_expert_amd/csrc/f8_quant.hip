// e4m3 quantisation, alone and behind an RMS norm: rows of bf16, fp16 or fp32 values into codes with an fp32 scale
// for each block of 128 (or 128 x 128) values; f8_device.h has the rules.
//
//   norm: h = x, or x + residual rounded to the type;  y_c = h_c w_c / sqrt(sum h^2 / cols + eps)
//
// All are one pass over memory, bound by it: 8192 x 8192 bf16 in 1 x 128 blocks 43 us, 4.7 TB/s.  A thread takes
// eight neighbouring values (16 or 32 bytes, the widest loads), so a block of 128 lies in 16 neighbouring lanes and
// its largest value is four lane moves away, without LDS.
#include "f8_device.h"
#include "f8_internal.h"

namespace qtip {

namespace {

constexpr int kPerThread = 8;

// Eight values at any element's address, as floats.
struct Bf16 {
  typedef uint16_t Elem;
  static __device__ float to_float(uint16_t e) { return f8_float((uint32_t)e << 16); }
  static __device__ uint16_t from_float(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct F16 {
  typedef uint16_t Elem;
  static __device__ float to_float(uint16_t e) { return (float)__builtin_bit_cast(_Float16, e); }
  static __device__ uint16_t from_float(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct F32 {
  typedef uint32_t Elem;
  static __device__ float to_float(uint32_t e) { return f8_float(e); }
  static __device__ uint32_t from_float(float v) { return f8_bits(v); }
};

template <class T>
struct __attribute__((packed, aligned(sizeof(typename T::Elem)))) Eight {
  typename T::Elem e[kPerThread];
};

// `left`: how many of the eight there are; the others count as zeros.
template <class T>
__device__ inline void load_eight(const void* base, int64_t at, int left, float (&v)[kPerThread]) {
  const typename T::Elem* src = reinterpret_cast<const typename T::Elem*>(base) + at;
  if (left >= kPerThread) {
    const Eight<T> w = *reinterpret_cast<const Eight<T>*>(src);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) v[i] = T::to_float(w.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) v[i] = i < left ? T::to_float(src[i]) : 0.0f;
  }
}

template <class T>
__device__ inline void store_eight(void* base, int64_t at, int left, const float (&v)[kPerThread]) {
  typename T::Elem* dst = reinterpret_cast<typename T::Elem*>(base) + at;
  if (left >= kPerThread) {
    Eight<T> w;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) w.e[i] = T::from_float(v[i]);
    *reinterpret_cast<Eight<T>*>(dst) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (i < left) dst[i] = T::from_float(v[i]);
  }
}

__device__ inline uint32_t top_of(const float (&v)[kPerThread]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) top = max(top, f8_bits(v[i]) & 0x7fffffffu);
  return top;
}

// Codes of eight values from column c on; a row's bytes end with zeros at a multiple of 16.
__device__ inline void store_codes(uint8_t* row, int64_t row_bytes, int64_t c, const float (&v)[kPerThread],
                                   const F8Scale& s) {
  if (c >= row_bytes) return;
  uint32_t codes[2];
  f8_codes(v, s, codes);
  *reinterpret_cast<uint2*>(row + c) = make_uint2(codes[0], codes[1]);
}

// ---- 1 x 128 blocks ----------------------------------------------------------------------------
constexpr int kQuantThreads = 256;

template <class T>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(F8QuantParams p) {
  const uint32_t blocks = ((uint32_t)p.cols + kF8Block - 1) / kF8Block;
  const int64_t item = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x;
  const uint32_t block = (uint32_t)(item >> 4);  // rows x blocks < 2^28
  if (block >= blocks * (uint32_t)p.rows) return;  // a block's 16 threads leave together
  const uint32_t row = block / blocks;
  const int64_t c = (int64_t)(block - row * blocks) * kF8Block + (item & 15) * kPerThread;
  float v[kPerThread];
  load_eight<T>(p.src, (int64_t)row * p.row_stride + c, (int)min((int64_t)kPerThread, p.cols - c), v);
  const F8Scale s(max_of_16(top_of(v)), p.pow2);
  const int64_t row_bytes = f8_row_bytes(p.cols);
  store_codes(p.codes + row * row_bytes, row_bytes, c, v, s);
  if ((item & 15) == 0) p.scales[block] = s.scale;
}

// ---- 128 x 128 blocks --------------------------------------------------------------------------
// A workgroup a block, its values in registers: 16 threads a row, each with two rows.  8192 x 8136 fp32: 69 us, 4.8 TB/s;
// with 256 threads of eight rows each 76, with 512 74: fewer waves have less asked for at a time.
constexpr int kTileThreads = 1024;
constexpr int64_t kMostTiles = UINT32_MAX / kTileThreads;  // of a launch, which has below 2^32 threads

template <class T>
__global__ __launch_bounds__(kTileThreads) void quantize_tile_kernel(F8QuantParams p) {
  constexpr int kRowsAtOnce = kTileThreads / 16, kSteps = kF8Block / kRowsAtOnce;
  __shared__ uint32_t tops[kTileThreads / 64];
  const uint32_t blocks = ((uint32_t)p.cols + kF8Block - 1) / kF8Block;
  const uint32_t block = p.first + blockIdx.x, br = block / blocks;  // below 2^24
  const int64_t c = (int64_t)(block - br * blocks) * kF8Block + (threadIdx.x & 15) * kPerThread;
  const int64_t row0 = (int64_t)br * kF8Block + (threadIdx.x >> 4);
  const int left = (int)min((int64_t)kPerThread, p.cols - c);
  float v[kSteps][kPerThread];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t row = row0 + i * kRowsAtOnce;
    load_eight<T>(p.src, row * p.row_stride + c, row < p.rows ? left : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) top = max(top, top_of(v[i]));
  top = max_of_16(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 64; ++i) top = max(top, tops[i]);
  const F8Scale s(top, p.pow2);
  const int64_t row_bytes = f8_row_bytes(p.cols);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t row = row0 + i * kRowsAtOnce;
    if (row < p.rows) store_codes(p.codes + row * row_bytes, row_bytes, c, v[i], s);
  }
  if (threadIdx.x == 0) p.scales[block] = s.scale;
}

template <class T>
void launch_quantize_type(F8QuantParams p, hipStream_t stream) {
  const int64_t blocks = ((int64_t)p.cols + kF8Block - 1) / kF8Block;
  if (p.block_rows == 1) {
    const int64_t grid = (blocks * 16 * p.rows + kQuantThreads - 1) / kQuantThreads;
    hipLaunchKernelGGL((quantize_rows_kernel<T>), dim3((unsigned)grid), dim3(kQuantThreads), 0, stream, p);
  } else {
    // many rows of few columns have more blocks than a launch: the next one takes them on
    const int64_t all = blocks * (((int64_t)p.rows + kF8Block - 1) / kF8Block);
    for (int64_t first = 0; first < all; first += kMostTiles) {
      p.first = (uint32_t)first;
      const int64_t grid = all - first < kMostTiles ? all - first : kMostTiles;
      hipLaunchKernelGGL((quantize_tile_kernel<T>), dim3((unsigned)grid), dim3(kTileThreads), 0, stream, p);
    }
  }
}

// ---- RMS norm ----------------------------------------------------------------------------------
// A workgroup a row.  Rows of up to kMaxHeld values stay in registers between the sum of squares and the norm
// (C chunks of eight a thread); longer ones are read again.  One chunk a thread where 1024 threads hold the row:
// 4096 x 8192 bf16 with the residual and the values 60 us (5.0 TB/s), two chunks of 512 threads 69; without a residual
// two chunks are the faster, 29.6 against 37 (683 x 8136 fp32: 10.5, 11.0).  16384 x 4096 108 us,
// 5.6 TB/s (some of it from the last-level cache); with the weights loaded ahead of the sum 117, registers that
// other rows could have used.  One row of 4096: 3.7 us, the chain of loads, sum, largest value and stores.
constexpr int kNormThreads = 1024;
constexpr int kMaxHeld = 4 * kPerThread * kNormThreads;

// The workgroup's sum of one value a thread, the same in all threads; order fixed by the launch's shape.
template <class V>
__device__ inline V sum_of_all(V v, V* partial) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  const int waves = (blockDim.x + 63) >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) partial[threadIdx.x >> 6] = v;
  __syncthreads();
  V sum = 0;
  for (int i = 0; i < waves; ++i) sum += partial[i];
  return sum;
}

struct NormFactor {
  float rstd;     // 1 / sqrt(mean + eps)
  double rstd64;  // the same where fp32's range does not hold the squares
  bool wide;
  __device__ float operator()(float h) const { return wide ? (float)((double)h * rstd64) : h * rstd; }
};

// `squares(as)` adds up this thread's squares in the type of its argument.
template <class F>
__device__ inline NormFactor norm_factor(const F8NormParams& p, F squares) {
  __shared__ float partial[kNormThreads / 64];
  __shared__ double partial64[kNormThreads / 64];
  const float sum = sum_of_all(squares(0.0f), partial);
  NormFactor f;
  f.rstd64 = 0.0;
  f.rstd = 1.0f / sqrtf(sum / (float)p.cols + p.eps);
  // Squares, or an eps, past fp32's range or next to its lower end (a NaN or an infinity comes here too and stays one)
  f.wide = !(sum < 0x1p126f) || p.eps > 0x1p126f || (sum < 0x1p-60f && sum != 0.0f) || (sum == 0.0f && p.eps < 0x1p-60f);
  if (f.wide) f.rstd64 = 1.0 / sqrt(sum_of_all(squares(0.0), partial64) / p.cols + (double)p.eps);
  return f;
}

__device__ inline void load_weight(const F8NormParams& p, int64_t c, int left, float (&w)[kPerThread]) {
  if (p.weight_type == kF8Bf16) load_eight<Bf16>(p.weight, c, left, w);
  else if (p.weight_type == kF8F16) load_eight<F16>(p.weight, c, left, w);
  else load_eight<F32>(p.weight, c, left, w);
}

// h of eight values from column c on, and its store where there is a residual.
template <class T>
__device__ inline void load_h(const F8NormParams& p, int64_t row, int64_t c, int left, float (&h)[kPerThread]) {
  load_eight<T>(p.x, row * p.x_stride + c, left, h);
  if (!p.residual) return;
  float r[kPerThread];
  load_eight<T>(p.residual, row * p.residual_stride + c, left, r);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) h[i] = T::to_float(T::from_float(h[i] + r[i]));
  store_eight<T>(p.residual_out, row * p.residual_stride + c, left, h);
}

template <class T>
__device__ inline void finish_eight(const F8NormParams& p, int64_t row, int64_t c, int left, const float (&h)[kPerThread],
                                    const NormFactor& f) {
  const int64_t blocks = ((int64_t)p.cols + kF8Block - 1) / kF8Block, row_bytes = f8_row_bytes(p.cols);
  float w[kPerThread], y[kPerThread];
  load_weight(p, c, left, w);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) y[i] = i < left ? f(h[i]) * w[i] : 0.0f;
  const F8Scale s(max_of_16(top_of(y)), p.pow2);
  store_codes(p.codes + row * row_bytes, row_bytes, c, y, s);
  if ((threadIdx.x & 15) == 0 && c < p.cols) p.scales[row * blocks + c / kF8Block] = s.scale;
  if (p.values && left > 0) store_eight<T>(p.values, row * p.cols + c, left, y);
}

template <class T, int C>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(F8NormParams p) {
  const int64_t row = blockIdx.x;
  float h[C][kPerThread];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * kPerThread;
    load_h<T>(p, row, c, (int)max(min((int64_t)kPerThread, p.cols - c), (int64_t)0), h[i]);
  }
  const NormFactor f = norm_factor(p, [&](auto sum) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) sum += (decltype(sum))h[i][j] * h[i][j];
    return sum;
  });
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * kPerThread;
    finish_eight<T>(p, row, c, (int)max(min((int64_t)kPerThread, p.cols - c), (int64_t)0), h[i], f);
  }
}

template <class T>
__global__ __launch_bounds__(kNormThreads) void norm_long_kernel(F8NormParams p) {
  const int64_t row = blockIdx.x;
  const int64_t chunks = ((int64_t)p.cols + kF8Block - 1) / kF8Block * (kF8Block / kPerThread);
  const void* again = p.residual ? p.residual_out : p.x;
  const int64_t stride = p.residual ? p.residual_stride : p.x_stride;
  bool first = true;  // the sums are stored once; a thread reads only what it wrote itself
  const NormFactor f = norm_factor(p, [&](auto zero) {
    // A thread adds up to 2^17 chunks one after the other: in fp64 (2^28 squares of 1.1 are 8e-4 off in fp32).
    double sum = 0.0;
    for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {
      const int left = (int)max(min((int64_t)kPerThread, p.cols - q * kPerThread), (int64_t)0);
      float h[kPerThread];
      if (first) load_h<T>(p, row, q * kPerThread, left, h);
      else load_eight<T>(again, row * stride + q * kPerThread, left, h);
      decltype(zero) eight = zero;
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) eight += (decltype(zero))h[j] * h[j];
      sum += eight;
    }
    first = false;
    return (decltype(zero))sum;
  });
  for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {  // whole blocks: 16 lanes stay together
    const int left = (int)max(min((int64_t)kPerThread, p.cols - q * kPerThread), (int64_t)0);
    float h[kPerThread];
    load_eight<T>(again, row * stride + q * kPerThread, left, h);
    finish_eight<T>(p, row, q * kPerThread, left, h, f);
  }
}

template <class T>
void launch_norm_type(const F8NormParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)p.rows);
  const int64_t chunks = ((int64_t)p.cols + kF8Block - 1) / kF8Block * (kF8Block / kPerThread);
  auto threads = [&](int c) { return dim3((unsigned)(((chunks + c - 1) / c + 63) / 64 * 64)); };
  if (p.cols <= 1 * kPerThread * kNormThreads)
    hipLaunchKernelGGL((norm_kernel<T, 1>), grid, threads(1), 0, stream, p);
  else if (p.cols <= 2 * kPerThread * kNormThreads)
    hipLaunchKernelGGL((norm_kernel<T, 2>), grid, threads(2), 0, stream, p);
  else if (p.cols <= kMaxHeld)
    hipLaunchKernelGGL((norm_kernel<T, 4>), grid, threads(4), 0, stream, p);
  else
    hipLaunchKernelGGL((norm_long_kernel<T>), grid, dim3(kNormThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_f8_quantize(const F8QuantParams& p, hipStream_t stream) {
  if (p.type == kF8Bf16) launch_quantize_type<Bf16>(p, stream);
  else if (p.type == kF8F16) launch_quantize_type<F16>(p, stream);
  else launch_quantize_type<F32>(p, stream);
  return hipGetLastError();
}

hipError_t launch_f8_rms_norm(const F8NormParams& p, hipStream_t stream) {
  if (p.type == kF8Bf16) launch_norm_type<Bf16>(p, stream);
  else if (p.type == kF8F16) launch_norm_type<F16>(p, stream);
  else launch_norm_type<F32>(p, stream);
  return hipGetLastError();
}

}  // namespace qtip
