// Device side of the MXFP4 quantisation: the rotation of a row held sixteen neighbouring columns
// per lane, and the encoding of those sixteen (x~ = P D^-1 x, then blocks of 32).
#pragma once

#include "mxfp4.h"

// The rotation's sums are defined as separately rounded fp32 operations (a fused multiply-add
// of the rescale and a butterfly would round differently from the definition).
#pragma clang fp contract(off)

namespace kq {
namespace {

constexpr int SPAN = 1024;       // columns that a wave holds: 16 neighbouring ones per lane

// Sixteen columns as they lie in memory (kept so until their turn: a conversion would wait for
// the load).
template <typename T>
struct Raw {
  u32x4 v[sizeof(T)];   // 16 columns: two words of bf16, four of fp32
  unsigned more;        // and, of a bf16 row that starts or ends inside a dword, the next dword
  int shift;            // and the bits of its first dword before the row
};

// The lane's columns c .. c + 15 of a row of n values, zero past its end: the descriptor ends with
// the row (at most 2^26 bytes).  WIDE: the row begins and ends with a dword (wide_rows; all rows of
// fp32).  Else the dwords that hold its first and last column are read whole and their other half
// is dropped (an 8794 x 28243 x with 384 output channels: 265 us; two bytes at a time 577).
template <bool WIDE>
__device__ __forceinline__ void load_columns(const float* row, int64_t c, int64_t n, Raw<float>& r) {
  const __amdgpu_buffer_rsrc_t rs = rsrc(row, (int)(4 * n));
#pragma unroll
  for (int k = 0; k < 4; ++k) r.v[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(4 * c) + 16 * k, 0, 0);
}
template <bool WIDE>
__device__ __forceinline__ void load_columns(const uint16_t* row, int64_t c, int64_t n, Raw<uint16_t>& r) {
  const int before = WIDE ? 0 : (int)((uintptr_t)row & 2);
  const __amdgpu_buffer_rsrc_t rs = rsrc((const uint8_t*)row - before, WIDE ? (int)(2 * n) : (int)(before + 2 * n + 2) & ~3);
#pragma unroll
  for (int k = 0; k < 2; ++k) r.v[k] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(2 * c) + 16 * k, 0, 0);
  if (!WIDE) {
    r.more = __builtin_amdgcn_raw_buffer_load_b32(rs, (int)(2 * c) + 32, 0, 0);
    r.shift = 8 * before;
  }
}

template <bool WIDE>
__device__ __forceinline__ void convert(const Raw<float>& w, int64_t c, int64_t n, float (&r)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) r[k] = __uint_as_float(w.v[k >> 2][k & 3]);
}
template <bool WIDE>
__device__ __forceinline__ void convert(const Raw<uint16_t>& w, int64_t c, int64_t n, float (&r)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    unsigned u = w.v[k >> 2][k & 3];
    if (!WIDE) u = __builtin_amdgcn_alignbit(k < 7 ? w.v[(k + 1) >> 2][(k + 1) & 3] : w.more, u, w.shift);
    r[2 * k] = __uint_as_float(u << 16);
    r[2 * k + 1] = __uint_as_float(u & 0xffff0000u);
  }
  if (!WIDE) {
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = c + k < n ? r[k] : 0.f;
  }
}

inline bool wide_rows(const MxRows& r) {
  return r.type == KQ_F32 || (((uintptr_t)r.x & 3) == 0 && r.ld % 2 == 0 && r.n % 2 == 0);
}

// The lane's factors sign / d of columns c .. c + 15, 1 past the last one.  WHOLE: d and the signs
// are 16-byte aligned and n is a multiple of 4 (whole_factors), so that a lane takes 16 bytes at a
// time (one column at a time, the lanes' loads are 64 bytes apart and cost more than a row's
// rotation).
template <bool WHOLE>
__device__ __forceinline__ void factors(const float* d, const int8_t* sign, int64_t c, int64_t n, float (&f)[16]) {
  const __amdgpu_buffer_rsrc_t rd = rsrc(d, d ? (int)(4 * n) : 0), rs = rsrc(sign, sign ? (int)n : 0);
  float dv[16];
  bool minus[16];
  if constexpr (WHOLE) {
    const u32x4 s = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)c, 0, 0);
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __builtin_amdgcn_raw_buffer_load_b128(rd, (int)(4 * c) + 16 * k, 0, 0);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      dv[k] = __uint_as_float(v[k >> 2][k & 3]);
      minus[k] = (s[k >> 2] >> (8 * (k & 3) + 7)) & 1;
    }
  } else {
    int sv[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      dv[k] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, (int)(4 * c) + 4 * k, 0, 0));
      sv[k] = (int8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, (int)c + k, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) minus[k] = sv[k] < 0;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) f[k] = c + k < n ? __fdiv_rn(minus[k] ? -1.f : 1.f, d ? dv[k] : 1.f) : 1.f;
}

__host__ __device__ inline bool whole_factors(const float* d, const int8_t* sign, int64_t n) {
  return (((uintptr_t)d | (uintptr_t)sign) & 15) == 0 && n % 4 == 0;
}

// The value of another lane (DPP: the move is part of the add that takes it).
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
// Holds sixteen values at this point of the program.
__device__ __forceinline__ void pin(float (&r)[16]) {
  asm volatile("" : "+v"(r[0]), "+v"(r[1]), "+v"(r[2]), "+v"(r[3]), "+v"(r[4]), "+v"(r[5]), "+v"(r[6]), "+v"(r[7]),
                    "+v"(r[8]), "+v"(r[9]), "+v"(r[10]), "+v"(r[11]), "+v"(r[12]), "+v"(r[13]), "+v"(r[14]), "+v"(r[15]));
}

// Butterflies of strides 1 .. 512 below the rotation block, 2^LOGH columns (LOGH < 0: `had`); of a
// block of S waves those below 64 S.
template <int LOGH>
__device__ __forceinline__ void span_stages(float (&r)[16], int had) {
  constexpr int XOR1 = 0xb1, XOR2 = 0x4e, XOR3 = 0x1b, HALF_MIRROR = 0x141, ROR8 = 0x128;
  const int lane = threadIdx.x & 63;
  auto on = [&](int h) { return LOGH < 0 ? had > h : (LOGH > 10 ? 64 << (LOGH - 10) : 1 << (LOGH < 0 ? 0 : LOGH)) > h; };
  auto up = [&](int bit) { return (unsigned)(lane & bit) << (31 - __builtin_ctz(bit)); };
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
    if (on(h)) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if ((k & h) == 0) {
          const float u = r[k], v = r[k | h];
          r[k] = u + v;
          r[k | h] = u - v;
        }
    }
  // Between lanes: the values with the upper lanes' signs turned, then each partner's added.  A lane
  // move waits for the instruction before it, so that each step is done for all sixteen.
  float x[16];
  auto turned = [&](int bit) {
    const unsigned u = up(bit);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(__float_as_uint(r[k]) ^ u);
    pin(x);
  };
  if (on(16)) {
    pin(r);
    turned(1);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = moved<XOR1>(r[k]) + x[k];
    pin(r);
  }
  if (on(32)) {
    turned(2);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = moved<XOR2>(r[k]) + x[k];
    pin(r);
  }
  if (on(64)) {   // lane xor 4 = (xor 7) xor 3
    turned(4);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = moved<HALF_MIRROR>(r[k]);
    pin(r);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = moved<XOR3>(r[k]) + x[k];
    pin(r);
  }
  if (on(128)) {
    turned(8);
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = moved<ROR8>(r[k]) + x[k];
    pin(r);
  }
  // Two values at a time: the exchange gives a lane both ends of one value's butterfly, a second
  // one hands the results back.
  if (on(256)) {
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const auto e = __builtin_amdgcn_permlane16_swap(__float_as_uint(r[k]), __float_as_uint(r[k + 1]), false, false);
      const float a = __uint_as_float(e[0]), b = __uint_as_float(e[1]);
      const auto f = __builtin_amdgcn_permlane16_swap(__float_as_uint(a + b), __float_as_uint(a - b), false, false);
      r[k] = __uint_as_float(f[0]);
      r[k + 1] = __uint_as_float(f[1]);
    }
  }
  if (on(512)) {
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const auto e = __builtin_amdgcn_permlane32_swap(__float_as_uint(r[k]), __float_as_uint(r[k + 1]), false, false);
      const float a = __uint_as_float(e[0]), b = __uint_as_float(e[1]);
      const auto f = __builtin_amdgcn_permlane32_swap(__float_as_uint(a + b), __float_as_uint(a - b), false, false);
      r[k] = __uint_as_float(f[0]);
      r[k + 1] = __uint_as_float(f[1]);
    }
  }
}

// LDS floats that wave_stages needs for a workgroup of `waves`.
constexpr int plane_floats(int waves) { return 4 * 64 * waves + 8; }
constexpr int rotate_floats(int waves) { return 4 * plane_floats(waves); }

// Butterflies of strides 64 S .. 512 S of a block of S waves (the workgroup holds WAVES / S
// blocks), through LDS: the lanes' columns are written side by side, read back sixteen that are
// 64 S apart, and written again.  The four quarters of each lane's sixteen lie in planes of their
// own, a quarter of 32 banks apart: single words are taken half a wave at a time, and its 32 lanes
// then reach 32 banks (no conflicts counted; planes 16 floats apart: 36 % of the LDS cycles, and
// 16384 x 8192 with blocks of 8192 99.3 us instead of 98.3).
template <int WAVES, int S>
__device__ __forceinline__ void wave_stages(float (&r)[16], float* v) {
  constexpr int PLANE = plane_floats(WAVES);
  static_assert(PLANE % 32 == 8, "two of a half wave's lanes would share a bank");
  const int t = threadIdx.x, base = t / (64 * S) * (SPAN * S) + t % (64 * S);
  auto at = [](int i) { return ((i >> 2) & 3) * PLANE + (i >> 4) * 4 + (i & 3); };
  __syncthreads();   // the row before has been read back
#pragma unroll
  for (int k = 0; k < 4; ++k) *(float4*)(v + k * PLANE + 4 * t) = make_float4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
  __syncthreads();
  float u[16];
#pragma unroll
  for (int p = 0; p < 16; ++p) u[p] = v[at(base + 64 * S * p)];
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int p = 0; p < 16; ++p)
      if ((p & h) == 0) {
        const float a = u[p], b = u[p | h];
        u[p] = a + b;
        u[p | h] = a - b;
      }
#pragma unroll
  for (int p = 0; p < 16; ++p) v[at(base + 64 * S * p)] = u[p];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 w = *(const float4*)(v + k * PLANE + 4 * t);
    r[4 * k] = w.x; r[4 * k + 1] = w.y; r[4 * k + 2] = w.z; r[4 * k + 3] = w.w;
  }
}

// Where 1 / sqrt(had) is 2^-k, the power k that `encode` takes off the exponents instead.
constexpr int exact_shift(int logh) { return logh > 0 && logh % 2 == 0 ? logh / 2 : 0; }

// The whole rotation of the lane's columns: factors, butterflies, and 1 / sqrt(had) unless encode
// has it.
template <int WAVES, int LOGH>
__device__ __forceinline__ void rotate(float (&r)[16], bool scaled, const float (&f)[16], int had, float isb, float* lds) {
  if (scaled) {
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] *= f[k];
  }
  span_stages<LOGH>(r, had);
  if constexpr (LOGH > 10) wave_stages<WAVES, 1 << (LOGH - 10)>(r, lds);
  if (LOGH >= 0 ? LOGH % 2 == 1 : had > 1) {
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] *= isb;
  }
}

// The largest magnitude (bits; of an infinity or NaN at least 0x7f800000) of the block of 32 that
// the lane and its neighbour hold.
__device__ __forceinline__ unsigned block_top(const float (&r)[16]) {
  float top = __builtin_fabsf(r[0]);
#pragma unroll
  for (int k = 1; k < 16; ++k) top = __builtin_elementwise_maximum(top, __builtin_fabsf(r[k]));   // NaN wins
  const unsigned b = __float_as_uint(top) & 0x7fffffffu;
  return max(b, (unsigned)__builtin_amdgcn_mov_dpp((int)b, 0xb1, 0xf, 0xf, true));
}

// The lane's sixteen codes, column c in the lowest nibble, of r 2^-SHIFT.  Two neighbouring lanes
// make a block: its scale (a NaN or infinity in it: 2^127, `bad`, codes zero); `four`: the scale
// bytes of the 128 columns that the lane's group of 8 lanes holds.
// A product with 2^-SHIFT is exact, and so is a conversion with the scale that much larger, unless
// the product is subnormal; it is rounded then, so it is computed where a block's largest value
// comes near that (its scale byte would be under 3: above, every subnormal rounds to zero).
template <int SHIFT>
__device__ __forceinline__ u32x2 encode(float (&r)[16], float& scale, bool& bad, int& four) {
  const int lane = threadIdx.x & 63;
  unsigned top = block_top(r);
  int shift = SHIFT;
  if (SHIFT > 0 && __any(top - 1 < ((SHIFT + 5u) << 23) - 1)) {
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] *= __uint_as_float((127u - SHIFT) << 23);
    top = block_top(r);
    shift = 0;
  }
  const int ex = (int)(top >> 23);
  bad = ex == 255;
  const int byte = bad ? 255 : max(ex - 2 - shift, 0);          // e + 127
  auto power = [](int b) { return __uint_as_float(b > 0 ? (unsigned)min(b, 254) << 23 : 0x00400000u); };
  scale = power(byte);
  const float over = power(byte + shift);
  u32x2 w = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], r[8 * k], r[8 * k + 1], over, 0);
    w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], r[8 * k + 2], r[8 * k + 3], over, 1);
    w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], r[8 * k + 4], r[8 * k + 5], over, 2);
    w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], r[8 * k + 6], r[8 * k + 7], over, 3);
    w[k] = bad ? 0 : w[k];
  }
  four = byte << (4 * (lane & 6));
  four |= __builtin_amdgcn_mov_dpp(four, 0x4e, 0xf, 0xf, true);
  four |= __builtin_amdgcn_mov_dpp(four, 0x141, 0xf, 0xf, true);
  return w;
}

}  // namespace
}  // namespace kq
