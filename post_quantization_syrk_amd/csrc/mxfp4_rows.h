// Device side of the MXFP4 quantisation: the rotation of a row held eight neighbouring columns
// per lane, and the encoding of those eight (x~ = P D^-1 x, then blocks of 32).
#pragma once

#include "mxfp4.h"

// The rotation's sums are defined as separately rounded fp32 operations (a fused multiply-add
// of the rescale and a butterfly would round differently from the definition).
#pragma clang fp contract(off)

namespace kq {
namespace {

constexpr int SPAN = 512;        // columns that a wave holds: 8 neighbouring ones per lane

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((unsigned)*p << 16); }

// The lane's columns c .. c + 7 of a row of n values, zero past its end, without a branch around
// the loads (where paths join the compiler waits for all of them).  WIDE: 16 bytes at a time, of a
// row that starts 16-byte aligned and ends with a whole dword (wide_rows).
template <typename T, bool WIDE>
__device__ __forceinline__ void load_columns(const T* row, int64_t c, int64_t n, float (&r)[8]) {
  if constexpr (WIDE) {
    // the descriptor ends with the row: n * 4 <= 2^26 bytes
    const __amdgpu_buffer_rsrc_t rs = rsrc(row, (int)(n * (int64_t)sizeof(T)));
    const int at = (int)(c * (int64_t)sizeof(T));
    const u32x4 u = __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0);
    if constexpr (sizeof(T) == 4) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, at + 16, 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        r[k] = __uint_as_float(u[k]);
        r[k + 4] = __uint_as_float(v[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        r[2 * k] = __uint_as_float(u[k] << 16);
        r[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    }
  } else {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = load1(row + min(c + k, n - 1));
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = c + k < n ? v[k] : 0.f;
  }
}

inline bool wide_rows(const MxRows& r) {
  return aligned16(r.x) && (r.type == KQ_F32 ? r.ld % 4 == 0 : r.ld % 8 == 0 && r.n % 2 == 0);
}

// The lane's factors sign / d of columns c .. c + 7, 1 past the last one.
__device__ __forceinline__ void factors(const float* d, const int8_t* sign, int64_t c, int64_t n, float (&f)[8]) {
  float dv[8];
  int sv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t at = min(c + k, n - 1);
    dv[k] = d ? d[at] : 1.f;
    sv[k] = sign ? sign[at] : 1;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = c + k < n ? __fdiv_rn(sv[k] < 0 ? -1.f : 1.f, dv[k]) : 1.f;
}

// Butterfly with the lane whose value comes in `with`: the lower lane's sum, the upper one's
// difference (lower minus upper); `up`: the sign bit on upper lanes.
template <int CTRL>
__device__ __forceinline__ float across(float v, float with, unsigned up) {
  const int w = __builtin_amdgcn_mov_dpp((int)__float_as_uint(with), CTRL, 0xf, 0xf, true);
  return __uint_as_float(w) + __uint_as_float(__float_as_uint(v) ^ up);
}

// Butterflies of strides 8 .. 256 below `had`: lanes 1 .. 32 apart.
__device__ __forceinline__ void lane_stages(float (&r)[8], int had, int lane) {
  constexpr int XOR1 = 0xb1, XOR2 = 0x4e, XOR3 = 0x1b, HALF_MIRROR = 0x141, ROR8 = 0x128;
  auto up = [&](int bit) { return (unsigned)(lane & bit) << (31 - __builtin_ctz(bit)); };
  if (had > 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = across<XOR1>(r[k], r[k], up(1));
  }
  if (had > 16) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = across<XOR2>(r[k], r[k], up(2));
  }
  if (had > 32) {   // lane xor 4 = (xor 7) xor 3
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int m = __builtin_amdgcn_mov_dpp((int)__float_as_uint(r[k]), HALF_MIRROR, 0xf, 0xf, true);
      r[k] = across<XOR3>(r[k], __uint_as_float(m), up(4));
    }
  }
  if (had > 64) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = across<ROR8>(r[k], r[k], up(8));
  }
  // Two values at a time: the exchange gives a lane both ends of one value's butterfly, a second
  // one hands the results back.
  if (had > 128) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const auto e = __builtin_amdgcn_permlane16_swap(__float_as_uint(r[k]), __float_as_uint(r[k + 1]), false, false);
      const float a = __uint_as_float(e[0]), b = __uint_as_float(e[1]);
      const auto f = __builtin_amdgcn_permlane16_swap(__float_as_uint(a + b), __float_as_uint(a - b), false, false);
      r[k] = __uint_as_float(f[0]);
      r[k + 1] = __uint_as_float(f[1]);
    }
  }
  if (had > 256) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const auto e = __builtin_amdgcn_permlane32_swap(__float_as_uint(r[k]), __float_as_uint(r[k + 1]), false, false);
      const float a = __uint_as_float(e[0]), b = __uint_as_float(e[1]);
      const auto f = __builtin_amdgcn_permlane32_swap(__float_as_uint(a + b), __float_as_uint(a - b), false, false);
      r[k] = __uint_as_float(f[0]);
      r[k + 1] = __uint_as_float(f[1]);
    }
  }
}

// Butterflies of strides 512 .. SPAN WAVES / 2 below `had`, between the workgroup's waves
// through LDS: the lanes' columns are written side by side (the two halves of each lane's eight
// in planes of their own, half the banks apart, so that neither access conflicts), read 512
// apart, eight per thread, and written back.  A block of 16 spans takes its last stage while
// the columns are read back.
template <int WAVES>
__device__ __forceinline__ void wave_stages(float (&r)[8], int had, float* v) {
  constexpr int PLANE = 4 * 64 * WAVES + 32;
  const int t = threadIdx.x;
  auto at = [](int i) { return ((i >> 2) & 1) * PLANE + (i >> 3) * 4 + (i & 3); };
  __syncthreads();   // the row before has been read back
  *(float4*)(v + 4 * t) = make_float4(r[0], r[1], r[2], r[3]);
  *(float4*)(v + PLANE + 4 * t) = make_float4(r[4], r[5], r[6], r[7]);
  __syncthreads();
  // the eight spans 8 (t / 512) + j, column t mod 512; with fewer spans per workgroup (4 waves),
  // two columns of four spans
  constexpr int S = WAVES < 8 ? WAVES : 8, P = 8 / S;
  float u[P][S];
  const int base = (t / (64 * S)) * (SPAN * S), col = t % (64 * S);
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < S; ++j) u[p][j] = v[at(base + SPAN * j + col + 64 * S * p)];
#pragma unroll
  for (int h = 1; h < S; h <<= 1)
    if (had > SPAN * h) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < S; ++j)
          if ((j & h) == 0) {
            const float a = u[p][j], b = u[p][j | h];
            u[p][j] = a + b;
            u[p][j | h] = a - b;
          }
    }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < S; ++j) v[at(base + SPAN * j + col + 64 * S * p)] = u[p][j];
  __syncthreads();
  const float4 lo = *(const float4*)(v + 4 * t), hi = *(const float4*)(v + PLANE + 4 * t);
  r[0] = lo.x; r[1] = lo.y; r[2] = lo.z; r[3] = lo.w;
  r[4] = hi.x; r[5] = hi.y; r[6] = hi.z; r[7] = hi.w;
  if constexpr (WAVES == 16) {   // had is 16 spans: with fewer, a workgroup has 8 waves
    const int o = 4 * (t ^ 512);
    const float4 a = *(const float4*)(v + o), b = *(const float4*)(v + PLANE + o);
    const unsigned up = (unsigned)(t & 512) << 22;
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = w[k] + __uint_as_float(__float_as_uint(r[k]) ^ up);
  }
}

// LDS floats that wave_stages needs.
constexpr int rotate_floats(int waves) { return 2 * (4 * 64 * waves + 32); }

// The whole rotation of the lane's columns: factors, butterflies, 1 / sqrt(had).
template <int WAVES, bool LONG>
__device__ __forceinline__ void rotate(float (&r)[8], bool scaled, const float (&f)[8], int had, float isb, float* lds) {
  if (scaled) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] *= f[k];
  }
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
    if (had > h) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if ((k & h) == 0) {
          const float u = r[k], v = r[k | h];
          r[k] = u + v;
          r[k | h] = u - v;
        }
    }
  lane_stages(r, had, threadIdx.x & 63);
  if (LONG) wave_stages<WAVES>(r, had, lds);
  if (had > 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] *= isb;
  }
}

// The lane's eight codes, column c in the lowest nibble.  Four neighbouring lanes make a block:
// its scale (a NaN or infinity in it: 2^127, `bad`, codes zero); `four`: the scale bytes of the
// 128 columns that the lane's row of 16 lanes holds.
__device__ __forceinline__ unsigned encode(const float (&r)[8], float& scale, bool& bad, int& four) {
  const int lane = threadIdx.x & 63;
  unsigned top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(r[k]) & 0x7fffffffu);
  top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));
  top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));
  const int ex = (int)(top >> 23);
  bad = ex == 255;
  const int byte = bad ? 255 : max(ex - 2, 0);          // e + 127
  scale = __uint_as_float(byte > 0 ? (unsigned)min(byte, 254) << 23 : 0x00400000u);
  unsigned w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[0], r[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[2], r[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[4], r[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[6], r[7], scale, 3);
  four = byte << (2 * (lane & 12));
  four |= __builtin_amdgcn_mov_dpp(four, 0x124, 0xf, 0xf, true);
  four |= __builtin_amdgcn_mov_dpp(four, 0x128, 0xf, 0xf, true);
  return bad ? 0 : w;
}

}  // namespace
}  // namespace kq
