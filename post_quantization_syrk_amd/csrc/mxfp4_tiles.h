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
  bool y_far;              // rows of y too far apart for 32-bit offsets inside a tile
  int64_t ldy;
};

// A product with few rows (mxfp4_few.hip): whether it is one, whether it quantises the rows of x
// itself, and its launch (not fused: the rows are quantised, at p.xc and p.xs).
bool mx_few(const ProductArgs& p);
bool mx_few_fused(const ProductArgs& p, const MxRows& x);
kq_status mx_few_product(const ProductArgs& p, const MxRows& x, int64_t block, bool fused, hipStream_t s);

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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
