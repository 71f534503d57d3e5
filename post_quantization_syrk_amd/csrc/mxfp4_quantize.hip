// MXFP4 quantisation of rows, with the input side of the incoherence processing folded in:
// x~ = P D^-1 x per row, P = blockdiag(Had_b) diag(S) / sqrt(b), then blocks of 32.
#include "mxfp4_rows.h"

#include <math.h>

#include <algorithm>

#pragma clang fp contract(off)

namespace kq {
namespace {

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
  int step;                // rows from one that a unit takes to its next
  bool whole;              // whole_factors
};

// Stores sixteen columns: whole dwords, and where they begin inside one its half and, at the end, the
// other half (10470 x 10810 bf16 with values: 136 us; two bytes at a time 322).
__device__ __forceinline__ void store_columns(uint16_t* to, const u32x4 (&o)[2]) {
  struct __attribute__((packed, aligned(4))) Four { u32x4 v; };
  struct __attribute__((packed, aligned(4))) Three { unsigned v[3]; };
  if (((uintptr_t)to & 2) == 0) {
    ((Four*)to)[0].v = o[0];
    ((Four*)to)[1].v = o[1];
    return;
  }
  unsigned w[7];
#pragma unroll
  for (int k = 0; k < 7; ++k) w[k] = __builtin_amdgcn_alignbit(o[(k + 1) >> 2][(k + 1) & 3], o[k >> 2][k & 3], 16);
  to[0] = (uint16_t)o[0][0];
  *(Four*)(to + 1) = Four{u32x4{w[0], w[1], w[2], w[3]}};
  *(Three*)(to + 9) = Three{{w[4], w[5], w[6]}};
  to[15] = (uint16_t)(o[1][3] >> 16);
}

// A wave holds SPAN columns, sixteen neighbouring ones per lane (half a block of 32: one lane move
// for its largest value, four strides of the rotation without any), and takes one row after
// another, the next one's load in flight.  Rotation blocks of up to SPAN columns stay inside a wave
// (its four waves work on their own); longer ones are a workgroup's, and pass through LDS once.
// Bound by HBM without a rotation (28672 x 8192 fp32 with values: 280-307 us, 5.0-5.5 TB/s) and by the
// vector instructions with a long one (16384 x 8192 bf16, block 8192: 98-104 us, 3.3-3.5 TB/s, and 121-125
// in front of a product); 2048 x 11008 bf16, block 256: 19 us, with values 27; one row of 4096: 4.1 us.
// LOGH: the rotation block, 2^LOGH columns (-1: any up to SPAN, decided at run time).
template <typename T, int LOGH, bool WIDE>
__global__ __launch_bounds__(LOGH > 10 ? 64 << (LOGH - 10) : 256) void mx_quantize_kernel(QuantArgs a) {
  constexpr bool LONG = LOGH > 10;
  constexpr int WAVES = LONG ? 1 << (LOGH > 10 ? LOGH - 10 : 0) : 4, COLS = LONG ? SPAN * WAVES : SPAN;
  __shared__ __attribute__((aligned(16))) float lds[LONG ? rotate_floats(WAVES) : 4];
  const int lane = threadIdx.x & 63;
  // the wave's, or workgroup's, columns and rows
  const unsigned unit = LONG ? blockIdx.x : blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t kp = mx_pad(a.n), c = (int64_t)(unit % a.chunks) * COLS + 16 * (LONG ? (int)threadIdx.x : lane);
  const int64_t r0 = unit / a.chunks;
  if (r0 >= a.rows) return;
  const bool live = c < kp, scaled = a.d || a.sign;
  float f[16];
  if (scaled) {
    if (a.whole)
      factors<true>(a.d, a.sign, c, a.n, f);
    else
      factors<false>(a.d, a.sign, c, a.n, f);
  }
  const T* x = (const T*)a.src + r0 * a.ld;
  Raw<T> next;
  load_columns<WIDE>(x, c, a.n, next);
  uint8_t* codes = a.codes + r0 * (kp / 2) + c / 2;
  uint8_t* scales = a.scales + ((c >> 7) * a.rows + r0) * 4;
  uint16_t* values = a.values + r0 * a.ldv + c;
  const int64_t step_x = a.step * a.ld, step_codes = a.step * (kp / 2), step_values = a.step * a.ldv;
  for (int64_t row = r0; row < a.rows; row += a.step) {
    float r[16];
    convert<WIDE>(next, c, a.n, r);
    x += row + a.step < a.rows ? step_x : 0;   // (the last row once more rather than a branch)
    load_columns<WIDE>(x, c, a.n, next);
    rotate<WAVES, LOGH>(r, scaled, f, a.had, a.isb, lds);
    float s;
    bool bad;
    int four;
    const u32x2 w = encode<exact_shift(LOGH)>(r, s, bad, four);
    if (live) {
      *(u32x2*)codes = w;
      if ((lane & 7) == 0) *(int*)scales = four;
      if (a.values) {
        u32x4 o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          o[k][0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], s, 0));
          o[k][1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], s, 1));
          o[k][2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], s, 2));
          o[k][3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], s, 3));
          if (bad) o[k] = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        }
        if (c + 16 <= a.n)
          store_columns(values, o);
        else
          for (int k = 0; k < 16; ++k)
            if (c + k < a.n) values[k] = (uint16_t)(o[k >> 3][(k >> 1) & 3] >> (16 * (k & 1)));
      }
    }
    codes += step_codes;
    scales += 4 * (int64_t)a.step;
    values += step_values;
  }
}

template <typename T, int LOGH, bool WIDE>
kq_status launch(QuantArgs a, hipStream_t s) {
  constexpr bool LONG = LOGH > 10;
  constexpr int WAVES = LONG ? 1 << (LOGH > 10 ? LOGH - 10 : 0) : 4, COLS = LONG ? SPAN * WAVES : SPAN;
  a.chunks = (int)ceil_div(mx_pad(a.n), COLS);
  // rows per unit (a wave, or a workgroup of a long block): all units on the card at once, so that
  // none is left over and the factors sign / d are computed once (16384 x 8192, one block a row:
  // 123 us; 16 rows per unit, a round and a third: 130)
  constexpr int RESIDENT = 4 * (WIDE && sizeof(T) == 2 ? 6 : 5);   // waves per compute unit, by registers
  const int64_t run = ceil_div(a.rows * a.chunks, (int64_t)device_cu_count() * RESIDENT / (LONG ? WAVES : 1));
  a.step = (int)ceil_div(a.rows, run);
  const int64_t units = a.step * (int64_t)a.chunks, grid = LONG ? units : ceil_div(units, 4);
  if (units > 0x7fffffff)
    return fail(KQ_ESHAPE, "MXFP4 quantisation: %lld rows of %lld values", (long long)a.rows, (long long)a.n);
  mx_quantize_kernel<T, LOGH, WIDE><<<dim3((unsigned)grid), dim3(64 * WAVES), 0, s>>>(a);
  KQ_LAUNCHED("mx_quantize_kernel");
  return KQ_OK;
}

// The block is a constant of the kernel (as a variable, its stages copy the sixteen values at every
// branch), but for bf16 rows that begin or end inside a dword with a short rotation, which is rare:
// one kernel for those up to SPAN.
template <typename T>
kq_status launch_block(const QuantArgs& a, bool wide, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (!wide) switch (a.had > SPAN || a.had == 1 ? __builtin_ctz(a.had) : -1) {
      case 0: return launch<T, 0, false>(a, s);
      case 11: return launch<T, 11, false>(a, s);
      case 12: return launch<T, 12, false>(a, s);
      case 13: return launch<T, 13, false>(a, s);
      default: return launch<T, -1, false>(a, s);
    }
  }
  switch (__builtin_ctz(a.had)) {
    case 0: return launch<T, 0, true>(a, s);
    case 1: return launch<T, 1, true>(a, s);
    case 2: return launch<T, 2, true>(a, s);
    case 3: return launch<T, 3, true>(a, s);
    case 4: return launch<T, 4, true>(a, s);
    case 5: return launch<T, 5, true>(a, s);
    case 6: return launch<T, 6, true>(a, s);
    case 7: return launch<T, 7, true>(a, s);
    case 8: return launch<T, 8, true>(a, s);
    case 9: return launch<T, 9, true>(a, s);
    case 10: return launch<T, 10, true>(a, s);
    case 11: return launch<T, 11, true>(a, s);
    case 12: return launch<T, 12, true>(a, s);
    default: return launch<T, 13, true>(a, s);
  }
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
  a.whole = whole_factors(r.d, r.sign, r.n);
  const bool wide = wide_rows(r);
  return r.type == KQ_F32 ? launch_block<float>(a, wide, s) : launch_block<uint16_t>(a, wide, s);
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
