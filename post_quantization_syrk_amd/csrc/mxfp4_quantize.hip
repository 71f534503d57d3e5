// MXFP4 quantisation of rows, with the input side of the incoherence processing folded in:
// x~ = P D^-1 x per row, P = blockdiag(Had_b) diag(S) / sqrt(b), then blocks of 32.
#include "mxfp4.h"

#include <math.h>

#include <algorithm>

// The rotation's sums are defined as separately rounded fp32 operations (a fused multiply-add
// of the rescale and a butterfly would round differently from the definition).
#pragma clang fp contract(off)

namespace kq {
namespace {

constexpr int SPAN = 512;        // columns that a wave holds: 8 neighbouring ones per lane

struct QuantArgs {
  const void* src;
  int64_t rows, n, ld;
  const float* d;
  const int8_t* sign;
  int had;
  float isb;               // 1 / sqrt(had)
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* values;        // or NULL
  int64_t ldv;
  int chunks;              // workgroups that share a row
  int run;                 // consecutive rows per workgroup
  bool v_wide;             // rows of values are 16-byte aligned
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((unsigned)*p << 16); }

__device__ __forceinline__ void load8(const float* p, float (&r)[8]) {
  const float4 u = *(const float4*)p, v = *(const float4*)(p + 4);
  r[0] = u.x; r[1] = u.y; r[2] = u.z; r[3] = u.w;
  r[4] = v.x; r[5] = v.y; r[6] = v.z; r[7] = v.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&r)[8]) {
  const u32x4 u = *(const u32x4*)p;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    r[2 * k] = __uint_as_float(u[k] << 16);
    r[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
  }
}

// The lane's columns c .. c + 7 of a row of n values, zero past its end.
template <typename T, bool WIDE>
__device__ __forceinline__ void load_columns(const T* row, int64_t c, int64_t n, float (&r)[8]) {
  if (WIDE && c + 8 <= n) {
    load8(row + c, r);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = c + k < n ? load1(row + c + k) : 0.f;
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

// A workgroup holds SPAN WAVES columns, eight neighbouring ones per lane, and takes `run` rows
// one after another; four lanes make a block of 32.  Rotation blocks of up to 512 columns stay
// inside a wave (DPP and lane swaps), longer ones pass through LDS once (LONG).
template <typename T, int WAVES, bool LONG, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void mx_quantize_kernel(QuantArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[LONG ? 2 * (4 * 64 * WAVES + 32) : 4];
  const int lane = threadIdx.x & 63;
  const int64_t kp = mx_pad(a.n), c = (int64_t)(blockIdx.x % a.chunks) * (SPAN * WAVES) + 8 * threadIdx.x;
  const int64_t r0 = (int64_t)(blockIdx.x / a.chunks) * a.run, r1 = min(r0 + a.run, a.rows);
  const bool live = c < kp;
  if (!LONG && !live) return;
  const bool scaled = a.d || a.sign;
  float f[8];
  if (scaled) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = a.sign && c + k < a.n && a.sign[c + k] < 0 ? -1.f : 1.f;
      if (a.d && c + k < a.n) f[k] = __fdiv_rn(f[k], a.d[c + k]);
    }
  }
  const T* x = (const T*)a.src;
  float r[8];
  load_columns<T, WIDE>(x + r0 * a.ld, c, a.n, r);
  for (int64_t row = r0; row < r1; ++row) {
    float next[8];
    if (row + 1 < r1) load_columns<T, WIDE>(x + (row + 1) * a.ld, c, a.n, next);
    if (scaled) {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] *= f[k];
    }
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
      if (a.had > h) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((k & h) == 0) {
            const float u = r[k], v = r[k | h];
            r[k] = u + v;
            r[k | h] = u - v;
          }
      }
    lane_stages(r, a.had, lane);
    if (LONG) wave_stages<WAVES>(r, a.had, lds);
    if (a.had > 1) {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] *= a.isb;
    }
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(r[k]) & 0x7fffffffu);
    top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true));
    top = max(top, (unsigned)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true));
    const int ex = (int)(top >> 23);
    const bool bad = ex == 255;
    const int byte = bad ? 255 : max(ex - 2, 0);          // e + 127
    const float s = __uint_as_float(byte > 0 ? (unsigned)min(byte, 254) << 23 : 0x00400000u);
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[0], r[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[2], r[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[4], r[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, r[6], r[7], s, 3);
    if (bad) w = 0;
    // four blocks' bytes: the 16 lanes of a row hold 128 columns
    int four = byte << (2 * (lane & 12));
    four |= __builtin_amdgcn_mov_dpp(four, 0x124, 0xf, 0xf, true);
    four |= __builtin_amdgcn_mov_dpp(four, 0x128, 0xf, 0xf, true);
    if (live) {
      *(unsigned*)(a.codes + row * (kp / 2) + c / 2) = w;
      if ((lane & 15) == 0) *(int*)(a.scales + ((c >> 7) * a.rows + row) * 4) = four;
      if (a.values) {
        u32x4 o;
        o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
        if (bad) o = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        uint16_t* out = a.values + row * a.ldv + c;
        if (a.v_wide && c + 8 <= a.n) {
          *(u32x4*)out = o;
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < a.n) out[k] = (uint16_t)(o[k >> 1] >> (16 * (k & 1)));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = next[k];
  }
}

template <typename T, bool WIDE>
kq_status launch(QuantArgs a, hipStream_t s) {
  // a workgroup's waves: those of one rotation block, at least four
  const int waves = a.had > 8 * SPAN ? 16 : a.had > 4 * SPAN ? 8 : 4;
  a.chunks = (int)ceil_div(mx_pad(a.n), SPAN * waves);
  // rows per workgroup: enough to share the factors sign / d and to write the scales' lines whole,
  // as long as every place on the card (eight waves per SIMD) has a workgroup
  const int64_t places = (int64_t)device_cu_count() * 32 / waves;
  a.run = (int)std::max<int64_t>(1, std::min<int64_t>(16, a.rows * a.chunks / (2 * places)));
  const int64_t grid = ceil_div(a.rows, a.run) * a.chunks;
  if (grid > 0x7fffffff)
    return fail(KQ_ESHAPE, "MXFP4 quantisation: %lld rows of %lld values", (long long)a.rows, (long long)a.n);
  const dim3 g((unsigned)grid), t(64 * waves);
  if (a.had <= SPAN)
    mx_quantize_kernel<T, 4, false, WIDE><<<g, t, 0, s>>>(a);
  else if (waves == 4)
    mx_quantize_kernel<T, 4, true, WIDE><<<g, t, 0, s>>>(a);
  else if (waves == 8)
    mx_quantize_kernel<T, 8, true, WIDE><<<g, t, 0, s>>>(a);
  else
    mx_quantize_kernel<T, 16, true, WIDE><<<g, t, 0, s>>>(a);
  KQ_LAUNCHED("mx_quantize_kernel");
  return KQ_OK;
}

}  // namespace

kq_status mx_check_rows(const char* fn, const MxRows& r, int64_t* block) {
  if (r.type != KQ_F32 && r.type != KQ_BF16) return fail(KQ_EINVAL, "%s: type %d of the rows", fn, r.type);
  if (r.rows < 0 || r.rows > MX_MAX_ROWS || r.n < 1 || r.n > MX_MAX_N)
    return fail(KQ_ESHAPE, "%s: %lld rows of %lld values", fn, (long long)r.rows, (long long)r.n);
  if (r.ld < r.n) return fail(KQ_ESHAPE, "%s: leading dimension %lld < %lld", fn, (long long)r.ld, (long long)r.n);
  if (r.rows > 0 && !r.x) return fail(KQ_EINVAL, "%s: NULL rows", fn);
  if ((uintptr_t)r.x & (r.type == KQ_F32 ? 3 : 1)) return fail(KQ_EINVAL, "%s: rows not aligned to their type", fn);
  if (r.had < 0) return fail(KQ_ESHAPE, "%s: negative Hadamard block", fn);
  const int64_t b = r.had != 0 ? r.had : (r.n & -r.n);
  if (r.had == 0 && b > 8192)
    return fail(KQ_ENOTIMPL, "%s: the automatic Hadamard block (the largest power of 2 dividing the "
                "width) exceeds 8192; pass a block of at most 8192", fn);
  if (!is_pow2(b) || b > 8192 || r.n % b != 0)
    return fail(KQ_ESHAPE, "%s: the Hadamard block must be a power of 2 (<= 8192) dividing the width", fn);
  *block = b;
  return KQ_OK;
}

kq_status mx_quantize(const MxRows& r, int64_t block, uint8_t* codes, uint8_t* scales, uint16_t* values,
                      int64_t ldv, hipStream_t s) {
  if (r.rows == 0) return KQ_OK;
  QuantArgs a;
  a.src = r.x; a.rows = r.rows; a.n = r.n; a.ld = r.ld; a.d = r.d; a.sign = r.sign;
  a.had = (int)block; a.isb = (float)(1.0 / sqrt((double)block));
  a.codes = codes; a.scales = scales; a.values = values; a.ldv = ldv;
  a.v_wide = aligned16(values) && ldv % 8 == 0;
  // rows that start 16 bytes aligned are read 16 bytes at a time
  const bool wide = aligned16(r.x) && r.ld % (r.type == KQ_F32 ? 4 : 8) == 0;
  if (r.type == KQ_F32) return wide ? launch<float, true>(a, s) : launch<float, false>(a, s);
  return wide ? launch<uint16_t, true>(a, s) : launch<uint16_t, false>(a, s);
}

}  // namespace kq

extern "C" kq_status kq_mxfp4_quantize(const void* src, int src_type, int64_t rows, int64_t n, int64_t ld,
                                       const float* d, const int8_t* sign, int64_t had, uint8_t* codes,
                                       uint8_t* scales, uint16_t* values_opt, int64_t ldv, void* stream) {
  using namespace kq;
  const MxRows r{src, src_type, rows, n, ld, nullptr, d, sign, had};
  int64_t block = 1;
  KQ_TRY(mx_check_rows("kq_mxfp4_quantize", r, &block));
  if (rows > 0 && (!codes || !scales)) return fail(KQ_EINVAL, "kq_mxfp4_quantize: NULL argument");
  if (!aligned16(codes) || !aligned16(scales))
    return fail(KQ_EINVAL, "kq_mxfp4_quantize: codes and scales must be 16-byte aligned");
  if (values_opt && ldv < n) return fail(KQ_ESHAPE, "kq_mxfp4_quantize: ldv %lld < %lld", (long long)ldv, (long long)n);
  if ((uintptr_t)values_opt & 1) return fail(KQ_EINVAL, "kq_mxfp4_quantize: values not aligned to their type");
  return mx_quantize(r, block, codes, scales, values_opt, ldv, as_stream(stream));
}
