// What the products of packed operands share: tiles over expert bins, the order of workgroups, loads to LDS and
// the stores of their results.  P is a product's parameters: m, n, offsets, sorted_pair, out, out_bf16.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

namespace qtip {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int64_t kMostThreads = UINT32_MAX;  // of a launch

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ inline uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// silu(g) u.  From exp(-g) = 2^126 on the reciprocal is 0 and the result -0: silu itself is under 2^-119 there.
__device__ inline float swiglu(float g, float u) { return g * __builtin_amdgcn_rcpf(1.0f + expf(-g)) * u; }

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
template <class P>
__device__ inline int tile_row(const P& p, int start, int len, int i) {
  if (i >= len) return -1;
  if (!p.offsets) return start + i;
  const int r = p.sorted_pair[start + i];
  return r >= 0 && r < p.m ? r : -1;
}

// Stores SPAN neighbouring outputs of row r from column c on: a whole vector where p.n is a multiple
// of SPAN (so that it lies in the row or past it, aligned); otherwise a vector at any element's address, and one by one
// at the row's end.
template <int SPAN, class P>
__device__ inline void store_bf16(const P& p, int r, int c, const float (&v)[SPAN]) {
  if (c >= p.n) return;
  uint32_t w[SPAN / 2];
#pragma unroll
  for (int i = 0; i < SPAN / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  __bf16* d = reinterpret_cast<__bf16*>(p.out) + (size_t)r * p.n + c;
  if (SPAN == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[SPAN / 2 - 2], w[SPAN / 2 - 1]);
  else *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
}

template <int SPAN, class P>
__device__ inline void store_f32(const P& p, int r, int c, const float (&v)[SPAN]) {
  if (c >= p.n) return;
  float* d = reinterpret_cast<float*>(p.out) + (size_t)r * p.n + c;
#pragma unroll
  for (int i = 0; i < SPAN; i += 4) *reinterpret_cast<float4*>(d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

template <class E, int SPAN>
struct __attribute__((packed, aligned(sizeof(E)))) Neighbours {
  E e[SPAN];
};

template <class E, int SPAN>
__device__ inline void store_neighbours(void* out, size_t o, const float (&v)[SPAN]) {
  Neighbours<E, SPAN> w;
#pragma unroll
  for (int i = 0; i < SPAN; ++i) w.e[i] = (E)v[i];
  *reinterpret_cast<Neighbours<E, SPAN>*>(reinterpret_cast<E*>(out) + o) = w;
}

template <int SPAN, class P>
__device__ inline void store_odd(const P& p, int r, int c, const float (&v)[SPAN]) {
  const size_t o = (size_t)r * p.n + c;
  if (p.n - c >= SPAN) {
    if (p.out_bf16) store_neighbours<__bf16>(p.out, o, v);
    else store_neighbours<float>(p.out, o, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < SPAN; ++i) {
    if (c + i >= p.n) break;
    if (p.out_bf16) reinterpret_cast<__bf16*>(p.out)[o + i] = (__bf16)v[i];
    else reinterpret_cast<float*>(p.out)[o + i] = v[i];
  }
}

constexpr int kXcds = 8;  // workgroups go round-robin over the XCDs of an MI355X, each with its own L2

// The tile (of activation rows) and row block (of weight rows) of a workgroup.  Expert tiles go to
// the XCDs in turn, a tile's row blocks all to one: its activations stay in that XCD's L2, and the
// tiles past the last one (the grid is sized for the most there can be) are spread evenly.  Dense
// products give each XCD a run of consecutive blocks, walked down columns of 8 tiles, so that the
// blocks running at a time share few operand rows.
template <class P>
__device__ inline void tile_of_block(const P& p, int tiles, int row_blocks, int b, int& tile, int& rb) {
  const int xcd = b % kXcds, i = b / kXcds;
  if (p.offsets) {
    tile = i / row_blocks * kXcds + xcd;
    rb = i % row_blocks;
    return;
  }
  const int padded = (tiles + kXcds - 1) / kXcds * kXcds;
  const int at = xcd * (padded / kXcds * row_blocks) + i;  // a bijection: the grid is padded * row_blocks
  const int column = at / (8 * row_blocks), in = at % (8 * row_blocks);
  tile = column * 8 + in % 8;
  rb = in / 8;
}

typedef __attribute__((address_space(3))) void lds_void;

constexpr uint32_t kNoRow = 0x80000000u;  // a byte offset past every buffer resource's range

template <int I> struct Step { static constexpr int value = I; };

__device__ inline __amdgpu_buffer_rsrc_t product_rsrc(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7fffffff, 0x00020000);
}

// Waits until at most FLY vector memory operations are outstanding and LDS operations are done.
template <int FLY>
__device__ inline void wait_loads() {
  static_assert(FLY < 64, "");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((FLY & 15) | (FLY >> 4) << 14 | 7 << 4);
  asm volatile("" ::: "memory");
}

__device__ inline void wave_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace

}  // namespace qtip
