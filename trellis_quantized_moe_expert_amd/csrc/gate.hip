// Routing of a batch to its experts with a gate: scores, a bias for the choice, group-limited
// top-k, weights.
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
// Two experts' c_e can lie closer together than fp32 resolves (the scores of a sigmoid crowd
// together, the bias is added on top), so the choice is made on fp64 values.
#include "mx_internal.h"
#include "qtip_internal.h"

#include <cmath>

namespace qtip {

namespace {

constexpr int kGateWaves = 4;  // tokens per workgroup, one wave each

__device__ inline double shfl_xor_f64(double v, int mask) { return __shfl_xor(v, mask, 64); }

// The wave's best (value descending, index ascending); every lane gets it.
__device__ inline void wave_best(double& v, int& i) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const double ov = shfl_xor_f64(v, off);
    const int oi = __shfl_xor(i, off, 64);
    if (ov > v || (ov == v && oi < i)) {
      v = ov;
      i = oi;
    }
  }
}

__global__ __launch_bounds__(kGateWaves * 64) void gate_kernel(GateParams p) {
  __shared__ double choice_s[kGateWaves][kMaxExperts];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kGateWaves + wv;
  if (t >= p.n) return;  // a wave uses its own part of choice_s only; no barrier follows
  double* choice = choice_s[wv];
  const float* row = p.logits + (size_t)t * p.E;
  const int E = p.E, k = p.k;

  float top = -INFINITY;  // softmax: the largest logit that is a number
  double sum = 0.0;
  if (!p.sigmoid) {
    for (int e = lane; e < E; e += 64) top = fmaxf(top, row[e]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  }
  // (l == top) also where both are +inf, so an infinite logit takes the whole weight
  auto score_of = [&](float l) -> double {
    if (p.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
    return l == top ? 1.0 : exp((double)l - (double)top);
  };
  if (!p.sigmoid) {
    for (int e = lane; e < E; e += 64) {
      const float l = row[e];
      if (l > -INFINITY) sum += score_of(l);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += shfl_xor_f64(sum, off);
  } else {
    sum = 1.0;
  }
  for (int e = lane; e < E; e += 64) {
    const float l = row[e];
    double c = -INFINITY;
    if (l > -INFINITY) {
      c = score_of(l) / sum;
      if (p.bias) c += (double)p.bias[e];
      if (!(c > -INFINITY)) c = -INFINITY;
    }
    choice[e] = c;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  if (p.groups > 1) {
    const int size = E / p.groups;
    double mine = -INFINITY;  // lane g: the value of group g
    for (int g = 0; g < p.groups; ++g) {
      double value = -INFINITY;
      int taken = -1;
      for (int r = 0; r < p.group_top; ++r) {
        double bv = -INFINITY;
        int bi = 0x7fffffff;
        for (int q = lane; q < size; q += 64)
          if (q != taken && choice[g * size + q] > bv) {
            bv = choice[g * size + q];
            bi = q;
          }
        wave_best(bv, bi);
        if (bv > -INFINITY) value = r == 0 ? bv : value + bv;
        taken = bi;
      }
      if (lane == g) mine = value;
    }
    uint64_t kept = 0;
    for (int r = 0; r < p.top_groups; ++r) {
      double bv = (kept >> lane) & 1 ? -INFINITY : mine;
      int bi = bv > -INFINITY ? lane : 0x7fffffff;
      wave_best(bv, bi);
      if (bi < p.groups) kept |= 1ull << bi;
    }
    for (int e = lane; e < E; e += 64)
      if (!((kept >> (e / size)) & 1)) choice[e] = -INFINITY;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }

  int sel = -1;  // lane j: the j-th choice
  for (int j = 0; j < k; ++j) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int e = lane; e < E; e += 64)
      if (choice[e] > bv) {
        bv = choice[e];
        bi = e;
      }
    wave_best(bv, bi);
    if (bi >= E) break;  // nothing is left
    if (lane == j) sel = bi;
    if (lane == (bi & 63)) choice[bi] = -INFINITY;  // the lane that reads it again
  }
  double s = 0.0;
  if (sel >= 0) s = score_of(row[sel]) / sum;
  double z = s;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) z += shfl_xor_f64(z, off);
  if (p.renormalise) s = z > 0.0 ? s / z : 0.0;
  if (lane < k) {
    p.topk_idx[(size_t)t * k + lane] = sel;
    p.topk_w[(size_t)t * k + lane] = (float)(s * (double)p.scale);
  }
}

}  // namespace

hipError_t launch_gate(const GateParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(gate_kernel, dim3((unsigned)((p.n + kGateWaves - 1) / kGateWaves)), dim3(kGateWaves * 64), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace qtip
