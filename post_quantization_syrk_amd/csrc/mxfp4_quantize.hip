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

constexpr int QT = 256;          // threads per workgroup

// Byte of the scale of (row r, block b) of a matrix of `rows` rows: four blocks' bytes make a
// dword, the dwords of all rows follow each other.
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t b, int64_t rows) {
  return ((b >> 2) * rows + r) * 4 + (b & 3);
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((unsigned)*p << 16); }

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
  int seg;                 // columns per workgroup: a multiple of 128 and of had
};

// One segment of one row per workgroup: rescale and sign into LDS, butterflies there (strides
// ascending), then each thread quantises 16 columns; two lanes share a block.
template <typename T>
__global__ __launch_bounds__(QT) void mx_quantize_kernel(QuantArgs a) {
  extern __shared__ __attribute__((aligned(16))) float v[];
  const int t = threadIdx.x;
  const int64_t kp = mx_pad(a.n);
  const int nseg = (int)((kp + a.seg - 1) / a.seg);
  const int64_t row = blockIdx.x / nseg;
  const int64_t c0 = (int64_t)(blockIdx.x % nseg) * a.seg;
  const int len = (int)(kp - c0 < a.seg ? kp - c0 : a.seg);
  const int live = (int)(a.n - c0 < len ? a.n - c0 : len);
  const T* x = (const T*)a.src + row * a.ld + c0;
  for (int c = t; c < len; c += QT) {
    float xv = 0.f;
    if (c < live) {
      xv = load1(x + c);
      if (a.d || a.sign) {
        float f = a.sign && a.sign[c0 + c] < 0 ? -1.f : 1.f;
        if (a.d) f = __fdiv_rn(f, a.d[c0 + c]);
        xv *= f;
      }
    }
    v[c] = xv;
  }
  __syncthreads();
  for (int h = 1; h < a.had; h <<= 1) {
    for (int p = t; p < live / 2; p += QT) {
      const int i = ((p & ~(h - 1)) << 1) | (p & (h - 1));
      const float u = v[i], w = v[i + h];
      v[i] = u + w;
      v[i + h] = u - w;
    }
    __syncthreads();
  }
  for (int g = t; g < len / 16; g += QT) {
    float r[16];
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      r[j] = v[16 * g + j];
      if (a.had > 1) r[j] *= a.isb;
      top = max(top, __float_as_uint(r[j]) & 0x7fffffffu);
    }
    top = max(top, (unsigned)__shfl_xor((int)top, 1));   // len / 16 is even: both lanes are here
    const int ex = (int)(top >> 23);
    const bool bad = ex == 255;
    const int code = bad ? 255 : max(ex - 2, 0);          // e + 127
    const float s = __uint_as_float(code > 0 ? (unsigned)min(code, 254) << 23 : 0x00400000u);
    unsigned w[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      w[q] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[q], r[8 * q], r[8 * q + 1], s, 0);
      w[q] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[q], r[8 * q + 2], r[8 * q + 3], s, 1);
      w[q] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[q], r[8 * q + 4], r[8 * q + 5], s, 2);
      w[q] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[q], r[8 * q + 6], r[8 * q + 7], s, 3);
      if (bad) w[q] = 0;
    }
    const int64_t c = c0 + 16 * g;
    *(uint2*)(a.codes + row * (kp / 2) + c / 2) = make_uint2(w[0], w[1]);
    if ((g & 1) == 0) a.scales[scale_at(row, c >> 5, a.rows)] = (uint8_t)code;
    if (a.values) {
      uint16_t* out = a.values + row * a.ldv + c;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const unsigned el = (w[j >> 3] >> (4 * (j & 7))) & 15u;
        const int m = el & 1, ee = (el >> 1) & 3;
        const float mag = ee ? (float)((2 + m) << (ee - 1)) * 0.5f : 0.5f * m;
        const float val = bad ? __uint_as_float(0x7fc00000u) : (el & 8 ? -mag : mag) * s;
        if (c + j < a.n) out[j] = (uint16_t)(__float_as_uint(val) >> 16);   // exact in bf16
      }
    }
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
  a.seg = (int)std::max<int64_t>(4096, block);
  const int64_t nseg = ceil_div(mx_pad(r.n), a.seg);
  if (r.rows * nseg > 0x7fffffff)
    return fail(KQ_ESHAPE, "MXFP4 quantisation: %lld rows of %lld values", (long long)r.rows, (long long)r.n);
  const size_t lds = sizeof(float) * (size_t)a.seg;
  if (r.type == KQ_F32)
    mx_quantize_kernel<float><<<dim3((unsigned)(r.rows * nseg)), dim3(QT), lds, s>>>(a);
  else
    mx_quantize_kernel<uint16_t><<<dim3((unsigned)(r.rows * nseg)), dim3(QT), lds, s>>>(a);
  KQ_LAUNCHED("mx_quantize_kernel");
  return KQ_OK;
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
