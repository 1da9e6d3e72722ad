// Internal declarations of the MXFP4 operators and the expert gate (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qtip {

// ---- gate (gate.hip) -------------------------------------------------------------------------
constexpr int kGateMaxGroups = 64;  // one lane of a wave per group

struct GateParams {
  const float* logits;  // [n][E]
  const float* bias;    // [E] or NULL
  int32_t n, E, k;
  int32_t sigmoid;      // 0: softmax over the token's E logits
  int32_t groups, top_groups, group_top;
  int32_t renormalise;
  float scale;
  int32_t* topk_idx;    // [n][k]
  float* topk_w;        // [n][k]
};

constexpr int kGateMaxBlocks = 512;  // blocks of tokens whose counts a binning workgroup adds up

struct GateBins {
  int32_t* counts;       // [E]
  int32_t* offsets;      // [E + 1]
  int32_t* sorted_pair;  // [n k]
  int32_t* tile_map;     // NULL, or [n k][3]
  int32_t* n_tiles;
  int32_t tile_m;
  int32_t* hist;         // [kGateMaxBlocks][E]: scratch of a call with more tokens than a workgroup takes
};

// bins NULL: the experts and weights only.
hipError_t launch_gate(const GateParams& p, const GateBins* bins, hipStream_t stream);
// The bins of experts that another kernel has chosen (p.n, p.E, p.k, p.topk_idx).
hipError_t launch_gate_bins(const GateParams& p, const GateBins& bins, hipStream_t stream);

// The weighted sum of a token's pairs that have an expert (H a multiple of 4).
hipError_t launch_combine_chosen(const float* y, const float* topk_w, const int32_t* topk_idx, int32_t E, int32_t n,
                                 int32_t k, int32_t H, void* out, int out_bf16, hipStream_t stream);

// ---- MXFP4 (mx_quant.hip, mx_matmul.hip) -----------------------------------------------------
constexpr int kMxBlock = 32;       // values that share one scale
constexpr int kMxBlockBytes = 16;  // their codes

enum MxSource { kMxBf16 = 0, kMxF16 = 1, kMxF32 = 2 };

struct MxQuantParams {
  const void* src;      // [rows][row_stride] of the source type
  int64_t row_stride;   // elements
  int32_t rows, cols;
  int32_t source;       // MxSource
  int32_t nearest;      // scale rule: 0 floor, 1 nearest
  uint8_t* codes;       // [rows][blocks * 16]
  uint8_t* scales;      // [rows][blocks]
  void* values;         // NULL, or [rows][cols] of the source type
};

hipError_t launch_mx_quantize(const MxQuantParams& p, hipStream_t stream);

// y[m][n] = sum over K of a[m][.] w[n][.], both operands MXFP4.  With offsets the rows are the
// pairs of expert bins: expert e owns pairs sorted_pair[offsets[e] .. offsets[e + 1]), pair p reads
// activation row p / a_div, multiplies expert e's matrix and writes output row p.  With w1 the
// result is silu(a w0^T) * (a w1^T).
struct MxMatmulParams {
  const uint8_t* a;
  const uint8_t* a_scale;
  const uint8_t* w0;
  const uint8_t* w0_scale;
  const uint8_t* w1;        // or NULL
  const uint8_t* w1_scale;
  const int32_t* offsets;      // [E + 1], or NULL: dense rows 0 .. m - 1
  const int32_t* sorted_pair;  // [m]
  int32_t E;       // matrices in w0 (and w1)
  int32_t a_div;
  int32_t a_rows;  // rows of a
  int32_t m;       // rows of y: dense rows, or pairs
  int32_t n;       // rows of one w matrix
  int32_t blocks;  // 32-value blocks of a row (K / 32)
  void* out;       // [m][n]
  int32_t out_bf16;
};

hipError_t launch_mx_matmul(const MxMatmulParams& p, hipStream_t stream);

// Whether the product's threads are few enough for a launch (a plan's expert passes always fit).
bool mx_matmul_fits(const MxMatmulParams& p);

}  // namespace qtip
