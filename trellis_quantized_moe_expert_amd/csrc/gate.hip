// Routing of a batch to its experts with a gate: scores, a bias for the choice, group-limited
// top-k, weights, and the bins of the chosen pairs.
//
//   s_e = 1 / (1 + exp(-l_e))              (sigmoid)   or   exp(l_e - max l) / sum exp(l - max l)
//   c_e = s_e + bias_e                     decides the choice only
//   value of a group of E / G consecutive experts = sum of its 1 or 2 largest c_e
//   the top_groups groups of the largest value stay; of their experts the k largest c_e are chosen
//   w_j = s_{e_j} [/ sum_i s_{e_i}] * scale
//
// Every choice is by (value descending, index ascending).  An expert whose logit is -inf or NaN,
// or whose c_e is -inf or NaN, is never chosen; a slot that no expert is left for holds the id -1
// and the weight 0.
//
// A token is worked on by LANES neighbouring lanes, each holding consecutive experts of one group
// in registers, so that an order of (lane, register) is the order of expert ids, a group's value
// is a reduction over its lanes and all groups' reductions run at once.
//
// The choice is the one that fp64 makes: two experts' c_e can lie closer together than fp32
// resolves (the scores of a sigmoid crowd together, the bias is added on top).  Scores and groups
// are fp64 throughout (a vector fp64 instruction takes 6.5 to 7 cycles).  The choice runs on c_e rounded
// to fp32, which keeps every order that it does not make equal: each lane sorts its experts, and
// pairs of lanes merge their best KL until all lanes hold the token's best KL in order.  Where two
// neighbours of that order (the best one left among them) are equal in fp32, the wave chooses again
// on the fp64 values.
//
// What bounds it: the issue of fp64 instructions, not memory.  16384 tokens of 256 experts, 8 choices
// from the best 4 of 8 groups, sigmoid with bias (16.8 MB of logits, 3.9 us at the copy rate) take 21.7 us
// in the gate and 9 in placing, where each of 256 workgroups adds up all blocks' counts out of L2; 28 to 29 for
// the call.  A wave of four tokens issues 1870 vector instructions, about 700 of them fp64 (half for the
// 16 sigmoids of a lane, half for the sort and the merges).  With the constants
// and lane masks of a loop over tokens kept in vector registers the kernel spilled and took 25.  Small
// batches are bound by launches and the latency of a chain of dependent steps: a token of 8 choices,
// routed and binned by one workgroup, 7; 683 tokens of 5 choices 5.5 and 7.
#include "mx_internal.h"
#include "qtip_internal.h"

#include <cmath>

namespace qtip {

namespace {

constexpr int kGateWaves = 16;

// ---- reductions over the LANES lanes of a token; every lane gets the result --------------------
template <int CTRL>
__device__ inline float row_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

template <int LANES>
__device__ inline float lanes_max(float v) {
  v = fmaxf(v, row_move<0x121>(v));  // rotations of the 16-lane row by 1, 2, 4, 8
  v = fmaxf(v, row_move<0x122>(v));
  v = fmaxf(v, row_move<0x124>(v));
  v = fmaxf(v, row_move<0x128>(v));
  if (LANES == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

template <int CTRL>
__device__ inline double row_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

template <int LANES>
__device__ inline double lanes_max(double v) {
  v = fmax(v, row_move<0x121>(v));
  v = fmax(v, row_move<0x122>(v));
  v = fmax(v, row_move<0x124>(v));
  v = fmax(v, row_move<0x128>(v));
  if (LANES == 64) {
    v = fmax(v, __shfl_xor(v, 16, 64));
    v = fmax(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

template <int LANES>
__device__ inline double lanes_sum(double v) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// What exp_f64 multiplies by, in scalar registers.  The empty statements keep the compiler from moving
// the constants out of a loop over tokens, where it kept them in vector registers and spilled those.
struct ExpTerms {
  double log2e, ln2_hi, ln2_lo, c[11];  // c[i] = 1 / (13 - i)!
  __device__ inline ExpTerms() {
    log2e = 1.4426950408889634;
    ln2_hi = -0x1.62e42fefa39efp-1;
    ln2_lo = -0x1.abc9e3b39803fp-56;
    double factorial = 6227020800.0;  // 13!
#pragma unroll
    for (int i = 0; i < 11; ++i) {
      c[i] = 1.0 / factorial;
      factorial /= 13 - i;
      asm volatile("" : "+s"(c[i]));
    }
    asm volatile("" : "+s"(log2e), "+s"(ln2_hi), "+s"(ln2_lo));
  }
};

// exp(x), -1100 <= x <= 0, to about one unit in the last place: x = k ln 2 + r, |r| <= ln 2 / 2, ln 2 in
// two parts, and the Taylor polynomial of exp(r) up to r^13 / 13! (the next term is under 2^-57).
__device__ inline double exp_f64(double x, const ExpTerms& m) {
  const double k = rint(x * m.log2e);
  double r = fma(k, m.ln2_hi, x);
  r = fma(k, m.ln2_lo, r);
  double y = m.c[0];
#pragma unroll
  for (int i = 1; i < 11; ++i) y = fma(y, r, m.c[i]);
  y = fma(y, r, 0.5);
  y = fma(y, r, 1.0);
  y = fma(y, r, 1.0);
  return ldexp(y, (int)k);
}

// 1 / d, d in [1, 2048]: the hardware's estimate and two Newton steps.
__device__ inline double recip_f64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(fma(-d, y, 1.0), y, y);
  return fma(fma(-d, y, 1.0), y, y);
}

// The sigmoid of a logit, from the exponential of its negative magnitude: nothing overflows, and low logits
// keep their scores down to the end of fp64's range.
__device__ inline double sigmoid_f64(float l, const ExpTerms& m) {
  const double e = exp_f64((double)fmaxf(-fabsf(l), -1100.0f), m);
  const double r = recip_f64(1.0 + e);
  return l < 0.0f ? e * r : r;
}

// A logit's part of a softmax, 0 below exp(-1100).  l == top also where both are infinite: such logits
// share the weight.
__device__ inline double softmax_part(float l, float top, const ExpTerms& m) {
  return l == top ? 1.0 : exp_f64(fmax((double)l - (double)top, -1100.0), m);
}

// How a gate's groups lie on the lanes (host arithmetic).
struct GateShape {
  int32_t lanes_per_group;  // a power of two
  int32_t per_lane;         // experts of a lane, at most Q
};

// Takes the experts of groups that are not among the top_groups best out of c (c[q]: expert e0 + q).
template <int LANES, int Q>
__device__ inline void keep_groups(const GateParams& p, const GateShape& gs, double (&c)[Q]) {
  const int lane = threadIdx.x & 63, l = lane & (LANES - 1), base = lane - l;
  double a = -INFINITY, b = -INFINITY;  // the two largest
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    b = fmax(b, fmin(a, c[q]));
    a = fmax(a, c[q]);
  }
  for (int off = 1; off < gs.lanes_per_group; off <<= 1) {
    const double oa = __shfl_xor(a, off, 64), ob = __shfl_xor(b, off, 64);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  const double value = p.group_top == 2 && b > -INFINITY ? a + b : a;
  const int g = l / gs.lanes_per_group;
  int ahead = 0;
  for (int h = 0; h < p.groups; ++h) {
    const double o = __shfl(value, base + h * gs.lanes_per_group, 64);
    ahead += o > value || (o == value && h < g);
  }
  if (g >= p.groups || ahead >= p.top_groups) {
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] = -INFINITY;
  }
}

// A choice value and its expert in one number that orders like (value descending, id ascending): the
// order-preserving bits of the fp32 value above 1023 - id, kept as a double so that the minimum and
// maximum of two are one instruction each (positive, its exponent never all ones, 0: no expert).
__device__ inline double make_key(float v, int e) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);  // -0 becomes 0
  const uint32_t order = u & 0x80000000u ? ~u : u | 0x80000000u;
  return __builtin_bit_cast(double, (uint64_t)order << 30 | (uint32_t)(kMaxExperts - 1 - e));
}

template <int Q>
__device__ __attribute__((always_inline)) inline void sort_descending(double (&v)[Q]) {  // odd-even merge sort
#pragma unroll
  for (int n = 1; n < Q; n *= 2)
#pragma unroll
    for (int k = n; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % n; j + k < Q; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < Q && (i + j) / (2 * n) == (i + j + k) / (2 * n)) {
            const double hi = fmax(v[i + j], v[i + j + k]), lo = fmin(v[i + j], v[i + j + k]);
            v[i + j] = hi;
            v[i + j + k] = lo;
          }
}

// Merges the best KL, in order, of the lanes `a` with those of other lanes (b) into the best KL of
// both; lost: the best key that has gone.
template <int KL>
__device__ __attribute__((always_inline)) inline void merge_best(double (&a)[KL], const double (&b)[KL], double& lost) {
#pragma unroll
  for (int i = 0; i < KL; ++i) {
    lost = fmax(lost, fmin(a[i], b[KL - 1 - i]));
    a[i] = fmax(a[i], b[KL - 1 - i]);  // falls, then rises: a bitonic sequence
  }
#pragma unroll
  for (int s = KL / 2; s >= 1; s /= 2)
#pragma unroll
    for (int i = 0; i < KL; ++i)
      if (!(i & s)) {
        const double hi = fmax(a[i], a[i + s]), lo = fmin(a[i], a[i + s]);
        a[i] = hi;
        a[i + s] = lo;
      }
}

// The choice among the keys v, by one token's lanes: id[i] of lane l is the choice l + i LANES, -1
// past the last.  Returns whether two neighbours in the order have the same fp32 value.
template <int LANES, int Q, int KL, int TURNS>
__device__ __attribute__((always_inline)) inline bool choose_sorted(int k, double (&v)[Q], int (&id)[TURNS]) {
  const int l = threadIdx.x & (LANES - 1);
  sort_descending<Q>(v);
  double a[KL], b[KL], lost = 0.0;
#pragma unroll
  for (int i = 0; i < KL; ++i) a[i] = i < Q ? v[i < Q ? i : 0] : 0.0;
  if (Q > KL) lost = v[KL < Q ? KL : 0];
  // each step's partner holds another set of lanes' best: within fours, halves of a row, rows
#pragma unroll
  for (int i = 0; i < KL; ++i) b[i] = row_move<0xB1>(a[i]);  // lanes 1 0 3 2
  merge_best<KL>(a, b, lost);
#pragma unroll
  for (int i = 0; i < KL; ++i) b[i] = row_move<0x4E>(a[i]);  // lanes 2 3 0 1
  merge_best<KL>(a, b, lost);
#pragma unroll
  for (int i = 0; i < KL; ++i) b[i] = row_move<0x141>(a[i]);  // mirrored in eight
  merge_best<KL>(a, b, lost);
#pragma unroll
  for (int i = 0; i < KL; ++i) b[i] = row_move<0x140>(a[i]);  // mirrored in sixteen
  merge_best<KL>(a, b, lost);
  if (LANES == 64) {
#pragma unroll
    for (int i = 0; i < KL; ++i) b[i] = __shfl_xor(a[i], 16, 64);
    merge_best<KL>(a, b, lost);
#pragma unroll
    for (int i = 0; i < KL; ++i) b[i] = __shfl_xor(a[i], 32, 64);
    merge_best<KL>(a, b, lost);
  }
  lost = lanes_max<LANES>(lost);
  bool close = false;
#pragma unroll
  for (int t = 0; t < TURNS; ++t) {
    const int j = l + t * LANES;
    double mine = a[0], next = KL > 1 ? a[1] : lost;
#pragma unroll
    for (int i = 1; i < KL; ++i) {
      const double after = i + 1 < KL ? a[i + 1 < KL ? i + 1 : 0] : lost;
      mine = j == i ? a[i] : mine;
      next = j == i ? after : next;
    }
    const uint64_t m = __builtin_bit_cast(uint64_t, mine), n = __builtin_bit_cast(uint64_t, next);
    id[t] = j < k && m != 0 ? kMaxExperts - 1 - (int)(m & (kMaxExperts - 1)) : -1;
    close |= j < k && n != 0 && (m ^ n) >> 30 == 0;
  }
  return close;
}

// The same on fp64 values (v[q]: expert e0 + q; -inf: not to be chosen), equal ones by id.
template <int LANES, int Q, int TURNS>
__device__ __attribute__((always_inline)) inline void choose_exact(int k, double (&v)[Q], int e0, int (&id)[TURNS]) {
  const int lane = threadIdx.x & 63, l = lane & (LANES - 1), base = lane - l;
  for (int j = 0; j < k; ++j) {
    double best = v[0];
    int at = 0;
#pragma unroll
    for (int q = 1; q < Q; ++q) {
      at = v[q] > best ? q : at;
      best = v[q] > best ? v[q] : best;
    }
    const double top = lanes_max<LANES>(best);
    const uint64_t holders = __ballot(best == top && best > -INFINITY) >> base & (~0ull >> (64 - LANES));
    const int first = holders != 0 ? __ffsll((unsigned long long)holders) - 1 : 0;
    const int e = __shfl(e0 + at, base + first, 64);
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
      if (j == l + i * LANES) id[i] = holders != 0 ? e : -1;
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = holders != 0 && l == first && q == at ? -INFINITY : v[q];
  }
}

__device__ inline __amdgpu_buffer_rsrc_t float_rsrc(const float* base, int count) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base), (short)0, count * 4, 0x00020000);
}

// Q floats from byte offset `at` on; zeros past the resource's range.
template <int Q>
__device__ inline void load_four(__amdgpu_buffer_rsrc_t r, int at, float (&v)[Q]) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int q = 0; q < Q; q += 4) {
    const f32x4 x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 4 * q, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[q + i] = x[i];
  }
}

// The fp64 values of the experts a lane holds, -inf for those not to be chosen (their groups among
// them); e0: its first expert.  Its token's logits are at byte `at` of `logits`.  top, inv: a softmax's
// largest logit and 1 / sum.
template <int LANES, int Q>
__device__ __attribute__((always_inline)) inline void token_values(const GateParams& p, const GateShape& gs,
                                                                   __amdgpu_buffer_rsrc_t logits, int at, const ExpTerms& m,
                                                                   int& e0, float& top, double& inv, double (&c)[Q]) {
  const __amdgpu_buffer_rsrc_t biases = float_rsrc(p.bias, p.bias ? p.E : 0);
  const int l = threadIdx.x & (LANES - 1);
  const int size = p.E / p.groups;
  const int g = l / gs.lanes_per_group, in = (l & (gs.lanes_per_group - 1)) * gs.per_lane;
  e0 = g * size + in;
  const int have = g < p.groups ? min(max(size - in, 0), gs.per_lane) : 0;

  // Logits and biases, all asked for before the first is used: places without an expert read the
  // next ones, or zeros where that would pass the end.
  float lg[Q], bias[Q];
  load_four<Q>(logits, at + 4 * e0, lg);
  load_four<Q>(biases, 4 * e0, bias);  // zeros without a bias (a range of no bytes)
  top = -INFINITY;
  inv = 1.0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    lg[q] = q < have && lg[q] > -INFINITY ? lg[q] : -INFINITY;  // NaN: not to be chosen
    top = fmaxf(top, lg[q]);
  }
  if (p.sigmoid) {
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] = sigmoid_f64(lg[q], m);
  } else {
    top = lanes_max<LANES>(top);
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const double part = softmax_part(lg[q], top, m);
      c[q] = lg[q] > -INFINITY ? part : 0.0;
      sum += c[q];
    }
    sum = lanes_sum<LANES>(sum);
    inv = sum > 0.0 ? recip_f64(sum) : 0.0;
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] *= inv;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    c[q] += (double)bias[q];
    c[q] = lg[q] > -INFINITY && c[q] > -INFINITY ? c[q] : -INFINITY;
  }
  if (p.groups > 1) keep_groups<LANES, Q>(p, gs, c);
}

// The logits of the wave's tokens.
template <int LANES>
__device__ inline __amdgpu_buffer_rsrc_t token_rows(const GateParams& p, int first) {
  return float_rsrc(p.logits + (size_t)first * p.E, min(64 / LANES, p.n - first) * p.E);
}

template <int TURNS> struct Ids { int id[TURNS]; };

// The exact choice from the logits again: rarely needed, and a call of its own so that the fp64 values
// need not outlive the first choice.
template <int LANES, int Q, int TURNS>
__device__ __attribute__((noinline)) Ids<TURNS> choose_again(GateParams p, GateShape gs, int first, int at) {
  double c[Q], inv;
  int e0;
  float top;
  Ids<TURNS> ids;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) ids.id[i] = -1;
  token_values<LANES, Q>(p, gs, token_rows<LANES>(p, __builtin_amdgcn_readfirstlane(first)), at, ExpTerms(), e0, top,
                         inv, c);
  choose_exact<LANES, Q, TURNS>(p.k, c, e0, ids.id);
  return ids;
}

template <int TURNS> struct Chosen { float logit[TURNS]; };
template <int TURNS> struct Shares { double part[TURNS]; };

// Below this sum of the chosen scores their quotients come from low_shares: 1 / sum could pass fp64's
// range, and scores under 2^-1022 have lost bits.  (Above it a score of fewer than 52 bits has a share
// under 2^-322, nothing in fp32 whatever the scale.)
constexpr double kLowSum = 0x1p-700;

// The chosen scores divided by their sum where that is below kLowSum, from the logits (-inf: none).  Both
// scores then go like exp(l), so the largest chosen logit takes the place of the softmax's largest one.
// If even its score, exp(largest - top) (a sigmoid: top = 0), is below exp(-745), all are 0.  A call of
// its own, as choose_again: it is rarely needed.
template <int LANES, int TURNS>
__device__ __attribute__((noinline)) Shares<TURNS> low_shares(Chosen<TURNS> x, float top) {
  const ExpTerms terms;
  float largest = x.logit[0];
#pragma unroll
  for (int i = 1; i < TURNS; ++i) largest = fmaxf(largest, x.logit[i]);
  largest = lanes_max<LANES>(largest);
  const bool some = (double)largest - (double)top >= -745.0;  // false for -inf - -inf
  Shares<TURNS> s;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const double part = exp_f64(fmax((double)x.logit[i] - (double)largest, -1100.0), terms);
    s.part[i] = some && x.logit[i] > -INFINITY ? part : 0.0;
    sum += s.part[i];
  }
  sum = lanes_sum<LANES>(sum);
#pragma unroll
  for (int i = 0; i < TURNS; ++i) s.part[i] = some ? s.part[i] / sum : 0.0;
  return s;
}

// Routes the wave's 64 / LANES tokens from token `first` on.  sel: their ids in LDS, k of each (NULL:
// not wanted).
template <int LANES, int Q, int KL>
__device__ __attribute__((always_inline)) inline void gate_tokens(const GateParams& p, const GateShape& gs, int first,
                                                                  int32_t* sel) {
  constexpr int kTurns = KL > LANES ? KL / LANES : 1;
  const int lane = threadIdx.x & 63, l = lane & (LANES - 1), sub = lane / LANES;
  const int t = first + sub;  // past the last token: the lanes work on zeros and store nothing
  const bool there = t < p.n;
  const int at = sub * p.E * 4;
  const __amdgpu_buffer_rsrc_t logits = token_rows<LANES>(p, first);
  const ExpTerms terms;
  int id[kTurns];
  float top;
  double inv;
  bool close;
  {
    double c[Q];
    int e0;
    token_values<LANES, Q>(p, gs, logits, at, terms, e0, top, inv, c);
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] = c[q] > -INFINITY ? make_key((float)c[q], e0 + q) : 0.0;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) id[i] = -1;
    close = choose_sorted<LANES, Q, KL, kTurns>(p.k, c, id);
  }
  if (__ballot(close)) {
    const Ids<kTurns> again = choose_again<LANES, Q, kTurns>(p, gs, first, at);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) id[i] = again.id[i];
  }

  // the weights, a choice a lane
  Chosen<kTurns> x;
  double s[kTurns], z = 0.0;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    x.logit[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(logits, at + 4 * max(id[i], 0), 0, 0));
    x.logit[i] = id[i] >= 0 ? x.logit[i] : -INFINITY;
    const double part = p.sigmoid ? sigmoid_f64(x.logit[i], terms) : softmax_part(x.logit[i], top, terms) * inv;
    s[i] = id[i] >= 0 ? part : 0.0;
    z += s[i];
  }
  if (p.renormalise) {
    z = lanes_sum<LANES>(z);
    const bool low = z < kLowSum;
    z = 1.0 / z;
    if (__ballot(low)) {
      const Shares<kTurns> shares = low_shares<LANES, kTurns>(x, p.sigmoid ? 0.0f : top);
#pragma unroll
      for (int i = 0; i < kTurns; ++i) s[i] = low ? shares.part[i] : s[i];
      z = low ? 1.0 : z;
    }
  } else {
    z = 1.0;
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int j = l + i * LANES;
    if (j < p.k) {
      if (sel) sel[sub * p.k + j] = id[i];
      if (there) {
        p.topk_idx[(size_t)t * p.k + j] = id[i];
        p.topk_w[(size_t)t * p.k + j] = (float)(s[i] * z * (double)p.scale);
      }
    }
  }
  if (sel) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// ---- bins ---------------------------------------------------------------------------------------
// A stable counting sort of all pairs by expert, a block of pairs a workgroup.  The blocks' counts
// of each expert lie in hist [B][E]; every workgroup adds them up itself, once for its own place
// behind the earlier blocks and once for the bins' offsets, which takes no launch between and no
// waiting of workgroups for each other.
struct BinLds {
  int32_t wave_cnt[kGateWaves][kMaxExperts];  // a wave's pairs of each expert, then their first place
  int32_t total[kMaxExperts];
  int32_t before[kMaxExperts];
  int32_t wave_sum[kGateWaves];
};

// Inclusive scan over the 1024 threads.
__device__ inline int block_scan(int x, int32_t* wave_sum) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(x, off, 64);
    if (lane >= off) x += up;
  }
  __syncthreads();
  if (lane == 63) wave_sum[wv] = x;
  __syncthreads();
  for (int w = 0; w < wv; ++w) x += wave_sum[w];
  return x;
}

// A lane's rank among the wave's lanes that hold the same expert e (< E; E: none), and their number.
__device__ inline void peers_of(int e, int bits, int& rank, int& group) {
  uint64_t peers = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t m = __ballot((e >> b) & 1);
    peers &= ((e >> b) & 1) ? m : ~m;
  }
  const int lane = threadIdx.x & 63;
  rank = __popcll(peers & (lane == 0 ? 0ull : ~0ull >> (64 - lane)));
  group = __popcll(peers);
}

// Places pairs [p0, p0 + count) (ids from `ids`, indexed by pair) of block b of `blocks`; hist NULL:
// there is one block, and its counts are counted here.  Run by 1024 threads.  BATCH: times 64 pairs of a
// wave whose ids are asked for before the first is used, and the first of which are kept for the second
// walk (683 tokens of 5 pairs by one workgroup: 7.0 us with 8, 7.6 where the second walk reads them
// again, 8.6 with 1; a token of 8, which has one load a wave anyway: 7.3 with 1, 7.7 with 8).
template <int BATCH>
__device__ __attribute__((always_inline)) inline void bin_block(const GateBins& o, const int32_t* ids, int E, int p0,
                                                                int count, const int32_t* hist, int blocks, int b,
                                                                BinLds& s) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int bits = 1;
  while ((1 << bits) <= E) ++bits;
  const int chunk = ((count + kGateWaves - 1) / kGateWaves + 63) & ~63;
  const int lo = wv * chunk, hi = min(count, lo + chunk);
  auto load = [&](int i0, int (&id)[BATCH]) {
#pragma unroll
    for (int r = 0; r < BATCH; ++r) {
      const int i = i0 + 64 * r + lane;
      id[r] = ids[p0 + min(i, hi - 1)];
      id[r] = i < hi && id[r] >= 0 && id[r] < E ? id[r] : E;
    }
  };
  int first[BATCH];  // kept for the second walk
  if (lo < hi) load(lo, first);
  for (int e = lane; e < E; e += 64) s.wave_cnt[wv][e] = 0;
  for (int e = tid; e < E; e += 1024) s.total[e] = s.before[e] = 0;
  // the wave's pairs in order, 64 at a time: step(place, expert or E)
  auto each = [&](auto step) {
    auto walk = [&](int i0, const int (&id)[BATCH]) {
#pragma unroll
      for (int r = 0; r < BATCH; ++r)
        if (i0 + 64 * r < hi) step(i0 + 64 * r + lane, id[r]);
    };
    if (lo < hi) walk(lo, first);
    for (int i0 = lo + 64 * BATCH; i0 < hi; i0 += 64 * BATCH) {
      int id[BATCH];
      load(i0, id);
      walk(i0, id);
    }
  };
  each([&](int, int e) {
    int rank, group;
    peers_of(e, bits, rank, group);
    if (e < E && rank == 0) s.wave_cnt[wv][e] += group;
  });
  __syncthreads();
  if (hist) {
    // four experts a thread where rows are whole vectors: the loads of a thread are then a batch or two
    auto add = [&](auto vector) {
      typedef decltype(vector) V;
      constexpr int kVec = sizeof(V) / 4;
      int width = 16;
      while (width * kVec < E) width <<= 1;
      const int e = (tid & (width - 1)) * kVec, parts = 1024 / width;
      if (e >= E || tid / width >= blocks) return;
      int total[kVec] = {}, before[kVec] = {};
      for (int r = tid / width; r < blocks; r += 16 * parts) {
        V h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)  // rows past the last read it again and do not count
          h[i] = *reinterpret_cast<const V*>(hist + (size_t)min(r + i * parts, blocks - 1) * E + e);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int* x = reinterpret_cast<const int*>(&h[i]);
          const int row = r + i * parts;
#pragma unroll
          for (int q = 0; q < kVec; ++q) {
            total[q] += row < blocks ? x[q] : 0;
            before[q] += row < b ? x[q] : 0;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kVec; ++q) {  // whole numbers: the order does not matter
        atomicAdd(&s.total[e + q], total[q]);
        atomicAdd(&s.before[e + q], before[q]);
      }
    };
    if (E % 4 == 0) add(int4{});
    else add(int{});
    __syncthreads();
  } else {
    if (tid < E) {
      int c = 0;
      for (int w = 0; w < kGateWaves; ++w) c += s.wave_cnt[w][tid];
      s.total[tid] = c;
    }
  }
  const int c = tid < E ? s.total[tid] : 0;
  const int incl = block_scan(c, s.wave_sum);
  if (tid < E) {
    int run = incl - c + s.before[tid];
    for (int w = 0; w < kGateWaves; ++w) {
      const int nw = s.wave_cnt[w][tid];
      s.wave_cnt[w][tid] = run;
      run += nw;
    }
    if (b == 0) {
      o.counts[tid] = c;
      o.offsets[tid] = incl - c;
      if (tid == E - 1) o.offsets[E] = incl;
    }
  }
  if (b == 0 && o.tile_map) {  // uniform over the workgroup
    const int nt = (c + o.tile_m - 1) / o.tile_m;
    const int tincl = block_scan(nt, s.wave_sum);
    for (int q = 0; q < nt; ++q) {
      int32_t* m = o.tile_map + 3 * (size_t)(tincl - nt + q);
      m[0] = tid;
      m[1] = incl - c + q * o.tile_m;
      m[2] = min(o.tile_m, c - q * o.tile_m);
    }
    if (tid == E - 1) *o.n_tiles = tincl;
  }
  __syncthreads();
  each([&](int i, int e) {
    int rank, group;
    peers_of(e, bits, rank, group);
    if (e < E) {
      const int pos = s.wave_cnt[wv][e] + rank;  // every lane reads before the lowest lane advances it
      o.sorted_pair[pos] = p0 + i;
      if (rank == 0) s.wave_cnt[wv][e] = pos + group;
    }
  });
}

enum GateMode { kGateOnly, kGateCount, kGateBin };

// W waves, the tokens [blockIdx.x * per_block, + per_block).
template <int LANES, int Q, int KL, int W, int MODE>
__global__ __launch_bounds__(W * 64) void gate_kernel(GateParams p, GateShape gs, GateBins o, int per_block) {
  constexpr int kTokens = 64 / LANES;  // of a wave
  static_assert(MODE != kGateBin || W == kGateWaves, "");
  __shared__ int32_t sel[MODE == kGateCount ? W : 1][kTokens * kMaxTopK];
  __shared__ int32_t count[MODE == kGateCount ? kMaxExperts : 1];
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t0 = blockIdx.x * per_block, t1 = min(p.n, t0 + per_block);
  if (MODE == kGateCount) {
    for (int e = threadIdx.x; e < p.E; e += W * 64) count[e] = 0;
    __syncthreads();
  }
  for (int t = t0 + wv * kTokens; t < t1; t += W * kTokens) {
    gate_tokens<LANES, Q, KL>(p, gs, t, MODE == kGateCount ? sel[wv] : nullptr);
    if (MODE == kGateCount) {
      const int pairs = min(t1 - t, kTokens) * p.k;
      for (int i = lane; i < pairs; i += 64)
        if (sel[wv][i] >= 0) atomicAdd(&count[sel[wv][i]], 1);
    }
  }
  if (MODE == kGateCount) {
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += W * 64) o.hist[(size_t)blockIdx.x * p.E + e] = count[e];
  }
  if (MODE == kGateBin) {
    __shared__ BinLds s;
    __syncthreads();  // the workgroup's stores of topk_idx are visible to all of it
    bin_block<1>(o, p.topk_idx, p.E, 0, p.n * p.k, nullptr, 1, 0, s);
  }
}

__global__ __launch_bounds__(kGateWaves * 64) void place_kernel(GateParams p, GateBins o, int per_block, int blocks) {
  __shared__ BinLds s;
  const int b = blockIdx.x;
  const int t0 = b * per_block, t1 = min(p.n, t0 + per_block);
  bin_block<8>(o, p.topk_idx, p.E, t0 * p.k, (t1 - t0) * p.k, blocks > 1 ? o.hist : nullptr, blocks, b, s);
}

// The counts of each block of tokens whose experts another kernel has chosen.
__global__ __launch_bounds__(kGateWaves * 64) void count_kernel(GateParams p, GateBins o, int per_block) {
  __shared__ int32_t count[kMaxExperts];
  const int t0 = blockIdx.x * per_block, t1 = min(p.n, t0 + per_block);
  for (int e = threadIdx.x; e < p.E; e += kGateWaves * 64) count[e] = 0;
  __syncthreads();
  for (int i = t0 * p.k + threadIdx.x; i < t1 * p.k; i += kGateWaves * 64) {
    const int e = p.topk_idx[i];
    if (e >= 0 && e < p.E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kGateWaves * 64) o.hist[(size_t)blockIdx.x * p.E + e] = count[e];
}

// Tokens of a block, at least `pass`, so that there are at most kGateMaxBlocks.
int block_tokens(int n, int pass) {
  const int64_t passes = ((int64_t)n + (int64_t)pass * kGateMaxBlocks - 1) / ((int64_t)pass * kGateMaxBlocks);
  return (int)(pass * passes);
}

// out[t] = sum_j w[t, j] y[t k + j], j ascending, fp32, over the pairs that have an expert: the rows of
// the others were not written.  A thread takes four neighbouring outputs; up to eight rows' loads are
// issued before their multiply-adds.
__global__ __launch_bounds__(256) void combine_chosen_kernel(const float* __restrict__ y, const float* __restrict__ w,
                                                             const int32_t* __restrict__ topk_idx, int32_t E,
                                                             int32_t n, int32_t k, int32_t H, void* __restrict__ out,
                                                             int out_bf16) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  const int h4 = H >> 2;
  const int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= (int64_t)n * h4) return;
  const int t = (int)(item / h4), c = (int)(item - (int64_t)t * h4) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < k; j0 += 8) {
    float4 v[8];
    float wt[8];
    bool in[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      in[i] = j0 + i < k && (uint32_t)topk_idx[(size_t)t * k + min(j0 + i, k - 1)] < (uint32_t)E;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in[i]) {
        wt[i] = w[(size_t)t * k + j0 + i];
        v[i] = *reinterpret_cast<const float4*>(y + ((size_t)t * k + j0 + i) * H + c);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in[i]) {
        acc.x = fmaf(wt[i], v[i].x, acc.x);
        acc.y = fmaf(wt[i], v[i].y, acc.y);
        acc.z = fmaf(wt[i], v[i].z, acc.z);
        acc.w = fmaf(wt[i], v[i].w, acc.w);
      }
  }
  const size_t o = (size_t)t * H + c;
  if (out_bf16)
    *reinterpret_cast<bf16x4*>(reinterpret_cast<uint16_t*>(out) + o) =
        bf16x4{(__bf16)acc.x, (__bf16)acc.y, (__bf16)acc.z, (__bf16)acc.w};
  else
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + o) = acc;
}

template <int LANES, int Q, int KL, int W>
hipError_t launch_waves(const GateParams& p, const GateShape& gs, const GateBins* o, hipStream_t stream) {
  constexpr int kPass = W * (64 / LANES);  // tokens of a workgroup at a time
  if (!o) {
    hipLaunchKernelGGL((gate_kernel<LANES, Q, KL, W, kGateOnly>), dim3((unsigned)((p.n + kPass - 1) / kPass)),
                       dim3(W * 64), 0, stream, p, gs, GateBins{}, kPass);
    return hipGetLastError();
  }
  const int per_block = block_tokens(p.n, kPass), blocks = (p.n + per_block - 1) / per_block;
  hipLaunchKernelGGL((gate_kernel<LANES, Q, KL, W, kGateCount>), dim3((unsigned)blocks), dim3(W * 64), 0, stream, p,
                     gs, *o, per_block);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)blocks), dim3(kGateWaves * 64), 0, stream, p, *o, per_block, blocks);
  return hipGetLastError();
}

// A batch of at most a token a wave of one workgroup, routed and binned by it.
template <int Q, int KL>
hipError_t launch_few(const GateParams& p, const GateShape& gs, const GateBins& o, hipStream_t stream) {
  hipLaunchKernelGGL((gate_kernel<64, Q, KL, kGateWaves, kGateBin>), dim3(1), dim3(kGateWaves * 64), 0, stream, p, gs,
                     o, kGateWaves);
  return hipGetLastError();
}

template <int Q, int KL>
hipError_t launch_list(const GateParams& p, const GateShape& gs16, const GateShape& gs64, const GateBins* o,
                       hipStream_t stream) {
  if (o && p.n <= kGateWaves) return launch_few<Q, KL>(p, gs64, *o, stream);
  if (Q <= 16 && gs16.per_lane <= 16) {
    if (Q == 4 && p.n <= 1024) {
      // a token a wave while that leaves every SIMD one: half the work in a row of four tokens a wave
      hipLaunchKernelGGL((gate_kernel<64, 4, KL, 4, kGateOnly>), dim3((unsigned)((p.n + 3) / 4)), dim3(256), 0, stream,
                         p, gs64, GateBins{}, 4);
      const hipError_t e = hipGetLastError();
      return e != hipSuccess || !o ? e : launch_gate_bins(p, *o, stream);
    }
    // Four tokens a wave.  Small workgroups spread a batch over the CUs; larger ones make fewer blocks
    // to add up when placing.
    if (p.n <= 4096) return launch_waves<16, 16, KL, 4>(p, gs16, o, stream);
    return launch_waves<16, 16, KL, kGateWaves>(p, gs16, o, stream);
  }
  return launch_waves<64, Q < 16 ? 16 : Q, KL, kGateWaves>(p, gs64, o, stream);
}

template <int Q>
hipError_t launch_lanes(const GateParams& p, const GateShape& gs16, const GateShape& gs64, const GateBins* o,
                        hipStream_t stream) {
  return p.k <= 8 ? launch_list<Q, 8>(p, gs16, gs64, o, stream) : launch_list<Q, kMaxTopK>(p, gs16, gs64, o, stream);
}

}  // namespace

hipError_t launch_gate_bins(const GateParams& p, const GateBins& bins, hipStream_t stream) {
  // one workgroup places up to 8192 pairs in less time than a second launch takes
  const int per_block = (int64_t)p.n * p.k <= 8192 ? p.n : block_tokens(p.n, 64);
  const int blocks = (p.n + per_block - 1) / per_block;
  if (blocks > 1) {
    hipLaunchKernelGGL(count_kernel, dim3((unsigned)blocks), dim3(kGateWaves * 64), 0, stream, p, bins, per_block);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)blocks), dim3(kGateWaves * 64), 0, stream, p, bins, per_block,
                     blocks);
  return hipGetLastError();
}

hipError_t launch_combine_chosen(const float* y, const float* topk_w, const int32_t* topk_idx, int32_t E, int32_t n,
                                 int32_t k, int32_t H, void* out, int out_bf16, hipStream_t stream) {
  const int64_t items = (int64_t)n * (H / 4);
  hipLaunchKernelGGL(combine_chosen_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, stream, y, topk_w,
                     topk_idx, E, n, k, H, out, out_bf16);
  return hipGetLastError();
}

hipError_t launch_gate(const GateParams& p, const GateBins* bins, hipStream_t stream) {
  int lanes_of_groups = 1;  // groups rounded up to a power of two
  while (lanes_of_groups < p.groups) lanes_of_groups <<= 1;
  const int size = p.E / p.groups;
  auto shape = [&](int lanes) {
    GateShape gs{};
    gs.lanes_per_group = lanes / lanes_of_groups;
    gs.per_lane = gs.lanes_per_group > 0 ? (size + gs.lanes_per_group - 1) / gs.lanes_per_group : 1 << 30;
    return gs;
  };
  // A whole wave a token in a batch of few, 16 lanes a token in larger ones where a lane then has at
  // most 16 experts.
  const GateShape gs16 = shape(16), gs64 = shape(64);
  if (gs64.per_lane <= 4) return launch_lanes<4>(p, gs16, gs64, bins, stream);
  if (gs64.per_lane <= 16) return launch_lanes<16>(p, gs16, gs64, bins, stream);
  return launch_lanes<32>(p, gs16, gs64, bins, stream);  // per_lane <= 2 * 1024 / 64
}

}  // namespace qtip
