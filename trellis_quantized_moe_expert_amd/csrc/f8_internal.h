// Internal declarations of the e4m3 operators (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qtip {

constexpr int kF8Block = 128;  // values of a row that share one scale

enum F8Type { kF8Bf16 = 0, kF8F16 = 1, kF8F32 = 2 };

// Bytes of a row of codes.
inline __host__ __device__ int64_t f8_row_bytes(int64_t cols) { return (cols + 15) / 16 * 16; }

struct F8QuantParams {
  const void* src;     // [rows][row_stride] of the source type
  int64_t row_stride;  // elements
  int32_t rows, cols;
  int32_t type;        // F8Type
  int32_t block_rows;  // 1 or 128
  int32_t pow2;        // scale rule
  uint8_t* codes;      // [rows][f8_row_bytes(cols)]
  float* scales;       // [ceil(rows / block_rows)][ceil(cols / 128)]
  uint32_t first;      // the 128 x 128 block that a launch begins with; launch_f8_quantize sets it
};

hipError_t launch_f8_quantize(const F8QuantParams& p, hipStream_t stream);

struct F8NormParams {
  const void* x;            // [rows][x_stride]
  int64_t x_stride;
  const void* residual;     // NULL, or [rows][residual_stride]
  void* residual_out;       // the sums, laid out as the residual
  int64_t residual_stride;
  const void* weight;       // [cols]
  int32_t rows, cols;
  int32_t type, weight_type;  // F8Type
  float eps;
  int32_t pow2;
  uint8_t* codes;           // [rows][f8_row_bytes(cols)]
  float* scales;            // [rows][ceil(cols / 128)]
  void* values;             // NULL, or [rows][cols] of the type
};

hipError_t launch_f8_rms_norm(const F8NormParams& p, hipStream_t stream);

// y[m][n] = sum over the 128-blocks b of K: a_scale[m][b] w_scale[n / 128][b] sum a[m][.] w[n][.].  With
// offsets the rows are the pairs of expert bins: expert e owns pairs sorted_pair[offsets[e] .. offsets[e + 1]),
// pair p reads activation row p / a_div, multiplies expert e's matrix and writes output row p.  With w1 the
// result is silu(a w0^T) * (a w1^T), and may leave as e4m3 codes with a scale for each 128 of a row.
struct F8MatmulParams {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* w0;
  const float* w0_scale;
  const uint8_t* w1;  // or NULL
  const float* w1_scale;
  const int32_t* offsets;      // [E + 1], or NULL: dense rows 0 .. m - 1
  const int32_t* sorted_pair;  // [m]
  int32_t E;       // matrices in w0 (and w1)
  int32_t a_div;
  int32_t m;       // rows of y: dense rows, or pairs
  int32_t n;       // rows of one w matrix
  int32_t k;       // bytes of a row, a multiple of 16
  void* out;       // [m][n]: bf16, fp32, or, where out_scale is not NULL, e4m3 codes
  int32_t out_bf16;
  float* out_scale;  // [m][n / 128]; only with w1 and n a multiple of 128
};

hipError_t launch_f8_matmul(const F8MatmulParams& p, hipStream_t stream);

// Whether the product's threads are few enough for a launch (a plan's expert passes always fit).
bool f8_matmul_fits(const F8MatmulParams& p);

}  // namespace qtip
