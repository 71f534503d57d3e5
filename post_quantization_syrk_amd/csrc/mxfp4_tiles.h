// Device side that the MXFP4 products share: their arguments, the tiles of y, types.
#pragma once

#include "mxfp4.h"

namespace kq {

// A product's arguments on the device.
struct ProductArgs {
  const uint8_t* xc;       // rows x pitch
  const uint8_t* xs;
  int64_t rows;            // rows of x
  const uint8_t* wc;       // experts x N x pitch
  const uint8_t* ws;
  int64_t N;
  int64_t pitch;           // bytes of a quantised row: Kp / 2
  int steps;               // Kp / 128
  const int32_t* index;    // slot -> row of x, or NULL: the slot itself
  const int32_t* offsets;  // experts + 1 first slots, or NULL: one layer, slots = rows
  int experts;
  int64_t slots;
  void* y;
  bool y_bf16;
  bool y_far;              // rows of y (or of the residual) too far apart for 32-bit offsets inside a tile
  int64_t ldy;
  int epi;                 // EPI_*; what it applies:
  int act;
  const float* bias;       // experts x N, or NULL
  const void* residual;    // or NULL
  bool r_bf16;
  int64_t ldr;
};

// What a product applies to its sums: nothing, act(sum + bias) + residual, or that with pairs of
// columns, act(sum + bias) * (other sum + its bias) + residual.  A gated layer's N rows are those of
// the gate, then as many others; its columns are taken in pairs, so that both of a pair lie in one
// lane (or two neighbouring ones): column v is row v / 2 of the half v % 2.
enum { EPI_NONE, EPI_PLAIN, EPI_GATED };

// Row of the layer, from the first row of a tile at column n0, of column n0 + r.
template <int EPI>
__device__ __forceinline__ int64_t layer_row(const ProductArgs& a, int n0, int64_t r) {
  const int64_t c = r < a.N - 1 - n0 ? r : a.N - 1 - n0;   // (past the last column: that one)
  return EPI == EPI_GATED ? (c & 1) * (a.N >> 1) + (c >> 1) : c;
}
// The first row of a tile at column n0, and the column of y where it begins.
template <int EPI>
__device__ __forceinline__ int first_row(int n0) {
  return EPI == EPI_GATED ? n0 >> 1 : n0;
}

// A product with few rows (mxfp4_few.hip): whether it is one, whether it quantises the rows of x
// itself, and its launch (not fused: the rows are quantised, at p.xc and p.xs).
bool mx_few(const ProductArgs& p);
bool mx_few_fused(const ProductArgs& p, const MxRows& x);
kq_status mx_few_product(const ProductArgs& p, const MxRows& x, int64_t block, bool fused, hipStream_t s);

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Slots [first, last) of expert e0 + lane (none past the last expert), for the lanes of a wave: the
// offsets cut to [0, slots] and each one below an earlier one raised to it, so that the ranges follow
// one another, and have no more tiles than slots / BM + experts, whatever the offsets hold.  `top`:
// the end of the experts before e0 (0 for none), moved on to that of these.
__device__ __forceinline__ void expert_ranges(const ProductArgs& a, int e0, int& top, int& first, int& last) {
  const int lane = threadIdx.x & 63, n = (int)a.slots;
  first = min(max(a.offsets[min(e0 + lane, a.experts)], 0), n);
  last = min(max(a.offsets[min(e0 + lane + 1, a.experts)], 0), n);
  if (__any(last < first || first < top)) {
    first = max(first, top);   // running maximum
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) first = max(first, __shfl_up(first, o));
    last = max(last, first);
  }
  top = __builtin_amdgcn_readlane(last, 63);
}

// v / (1 + exp(-u)).  The product u log2 e rounds by 2^-24 of itself, a relative error of |u| 2^-24 in
// the exponential; the sigmoid moves by at most 0.23 times that (u s (1 - s) <= 0.23).
__device__ __forceinline__ float sigmoid_times(float v, float u) {
  return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * u));
}
// v Phi(v), Phi the normal distribution: with a = |v|, Phi(-a) = 2^-(a^2 log2(e) / 2 + r(a)), where r
// grows slowly, from 1 at 0 to 3.9 at 6.  The polynomial is r's, fitted over [0, 6] for the least
// error of v Phi(v) relative to v (2.4 roundings); past 6, where Phi(-a) < 2^-29, r(6) serves.  Relative
// to the result, which vanishes there, the error grows to 3e-5 at -3, 1e-3 at -4, 2e-2 at -5 and 0.2 at -6;
// that of 1 + erf in fp32 to 1e-5, 5e-4, 5e-2 and 1.
__device__ __forceinline__ float gelu(float v) {
  const float a = fabsf(v), t = fminf(a, 6.f);
  float r = fmaf(-8.4700869e-06f, t, 5.3903324e-05f);
  r = fmaf(r, t, 4.2123639e-04f);
  r = fmaf(r, t, -7.3892716e-03f);
  r = fmaf(r, t, 5.2691109e-02f);
  r = fmaf(r, t, -2.6219437e-01f);
  r = fmaf(r, t, 1.1511109f);
  r = fmaf(r, t, 0.99999988f);
  const float tail = __builtin_amdgcn_exp2f(-fmaf(a * a, 0.72134752f, r));
  return v * (v < 0.f ? tail : 1.f - tail);
}
// act of C values, the same act for every lane.
template <int C>
__device__ __forceinline__ void activate(int act, float (&v)[C]) {
  if (act == KQ_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = sigmoid_times(v[i], v[i]);
  } else if (act == KQ_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
  } else if (act == KQ_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = gelu(v[i]);
  } else if (act == KQ_ACT_GELU_TANH) {   // 1 + tanh(u) = 2 / (1 + exp(-2 u))
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = sigmoid_times(v[i], v[i] * fmaf(0.0713548163f * v[i], v[i], 1.59576912f));
  }
}

// Rows [m0, last) of y with expert e's layer, columns from n0: one tile.
struct Tile {
  int e, m0, last, n0;
};

// The expert of row tile mt, counted over the experts, and the tile's rows; false past the last.
template <int BM>
__device__ __forceinline__ bool search_rows(const ProductArgs& a, int mt, Tile& t) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0, top = 0; e0 < a.experts; e0 += 64) {
    int first, last;
    expert_ranges(a, e0, top, first, last);
    const int c = (last - first + BM - 1) / BM;
    int sum = c;   // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o);
      if (lane >= o) sum += v;
    }
    const int all = __builtin_amdgcn_readlane(sum, 63);
    if (mt < all) {
      const int src = __ffsll((unsigned long long)__ballot(sum > mt)) - 1;
      t.e = __builtin_amdgcn_readfirstlane(e0 + src);
      t.m0 = __builtin_amdgcn_readfirstlane(__shfl(first, src) + (mt - __shfl(sum - c, src)) * BM);
      t.last = __builtin_amdgcn_readfirstlane(__shfl(last, src));
      return true;
    }
    mt -= all;
  }
  return false;
}

// Zeros that copies of rows outside x read.
__device__ __attribute__((aligned(16))) uint32_t g_zeros[4];

__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(unsigned, bf16x2{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

}  // namespace
}  // namespace kq
