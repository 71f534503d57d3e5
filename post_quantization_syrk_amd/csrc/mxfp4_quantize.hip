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
  int run;                 // consecutive rows per workgroup
  bool v_wide;             // rows of values are 16-byte aligned
};

// A workgroup holds SPAN WAVES columns, eight neighbouring ones per lane, and takes `run` rows
// one after another; four lanes make a block of 32.  Rotation blocks of up to 512 columns stay
// inside a wave (DPP and lane swaps), longer ones pass through LDS once (LONG).
template <typename T, int WAVES, bool LONG, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void mx_quantize_kernel(QuantArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[LONG ? rotate_floats(WAVES) : 4];
  const int lane = threadIdx.x & 63;
  const int64_t kp = mx_pad(a.n), c = (int64_t)(blockIdx.x % a.chunks) * (SPAN * WAVES) + 8 * threadIdx.x;
  const int64_t r0 = (int64_t)(blockIdx.x / a.chunks) * a.run, r1 = min(r0 + a.run, a.rows);
  const bool live = c < kp;
  if (!LONG && !live) return;
  const bool scaled = a.d || a.sign;
  float f[8];
  if (scaled) factors(a.d, a.sign, c, a.n, f);
  const T* x = (const T*)a.src;
  float r[8];
  load_columns<T, WIDE>(x + r0 * a.ld, c, a.n, r);
  for (int64_t row = r0; row < r1; ++row) {
    float next[8];
    if (row + 1 < r1) load_columns<T, WIDE>(x + (row + 1) * a.ld, c, a.n, next);
    rotate<WAVES, LONG>(r, scaled, f, a.had, a.isb, lds);
    float s;
    bool bad;
    int four;
    const unsigned w = encode(r, s, bad, four);
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
  const bool wide = wide_rows(r);
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
