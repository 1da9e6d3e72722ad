// e4m3 codes with an fp32 scale a block: what the quantisations and the products' 8-bit epilogue share.
//
//   amax rule: scale = amax / 448 rounded to fp32      (448 = 1.75 * 2^8, the largest code)
//   pow2 rule: scale = the smallest power of two that is no less than amax / 448
//   both at least 2^-126, so that 1 / scale is an fp32 number
//   code = the e4m3 value nearest to x / scale, a tie the even one
//
// |x| / scale is at most 448 (1 + 2^-23), which rounds to 448: no code needs to be cut.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace qtip {

__device__ inline uint32_t f8_bits(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ inline float f8_float(uint32_t b) { return __builtin_bit_cast(float, b); }

// The largest of 16 neighbouring lanes' values (lanes 16 i .. 16 i + 15), in all of them.
__device__ inline uint32_t max_of_16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // quad lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // quad lanes 2 3 0 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // 7 - i of each 8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // 15 - i
  return v;
}

// A block's scale, from the bits of its largest magnitude; NaN where that is no number.
struct F8Scale {
  float scale, inverse;
  bool bad;    // NaN or infinity in the block: scale NaN, zero codes
  bool exact;  // x * inverse is x / scale exactly

  __device__ F8Scale(uint32_t top, bool pow2) {
    bad = top >= 0x7f800000u;
    exact = pow2;
    if (pow2) {
      const int field = max((int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
      scale = f8_float((uint32_t)field << 23);
      inverse = f8_float((uint32_t)(254 - field) << 23);
    } else {
      // amax / 448, correctly rounded: one step of Newton's on the product with the rounded inverse
      const float amax = f8_float(top), r = 1.0f / 448.0f;
      float q = amax * r;
      q = fmaf(fmaf(-448.0f, q, amax), r, q);
      scale = fmaxf(q, 0x1p-126f);
      inverse = __builtin_amdgcn_rcpf(scale);
    }
    if (bad) scale = f8_float(0x7fc00000u);
  }
};

// q, within 4 units of its last place of x / scale, moved to where it rounds as x / scale does: a border
// between two codes has its low 19 bits clear, so only a q next to such a number can be on the wrong side.
__device__ inline float f8_settle(float q, float x, float scale) {
  const uint32_t up = f8_bits(q) + 4;
  if ((up & 0x7ffffu) >= 8) return q;
  const float border = f8_float(up & ~0x7ffffu);
  if (scale < 0x1p-60f) {  // far from the end of fp32: the difference's sign must not be lost
    x *= 0x1p64f;
    scale *= 0x1p64f;
  }
  const float off = fmaf(-border, scale, x);
  if (off == 0.0f) return border;
  const bool away = (off > 0.0f) == !(f8_bits(border) >> 31);
  return f8_float(f8_bits(border) + (away ? 1u : ~0u));
}

// Codes of N values (a multiple of 4), four to a dword.  The products with the rounded inverse are within
// 2 units of the last place.  A wave looks again where one of its values is next to a number with its low 19 bits
// clear: a border (about one value in 65536), but also a code, zero among them.  By the amax rule a block's largest
// value is next to 448, so all waves look again; by powers of two the products are exact and none does.
template <int N>
__device__ inline void f8_codes(const float (&x)[N], const F8Scale& s, uint32_t (&codes)[N / 4]) {
  float q[N];
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = x[i] * s.inverse;
  if (!s.exact) {
    uint32_t near = ~0u;
#pragma unroll
    for (int i = 0; i < N; ++i) near = min(near, (f8_bits(q[i]) + 4) & 0x7ffffu);
    if (near < 8) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = f8_settle(q[i], x[i], s.scale);
    }
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    int c = 0;
    c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], c, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], c, true);
    codes[i] = s.bad ? 0u : (uint32_t)c;
  }
}

}  // namespace qtip
