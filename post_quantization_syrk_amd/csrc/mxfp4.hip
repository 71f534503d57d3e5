// Microscaled 4-bit floating point (MXFP4): quantisation of rows with the input side of the
// incoherence processing folded in, and the products of quantised activations with quantised
// layers (one layer, or one of many per row: a mixture's experts).
//
// A row of n values is held in blocks of 32: a scale 2^e per block and one E2M1 element per
// value.  With a the block's largest magnitude,
//   e = max(floor(log2 a) - 2, -127),   element = x / 2^e rounded to nearest, ties to even,
// on {0, 0.5, 1, 1.5, 2, 3, 4, 6}, magnitudes above 6 to 6.  A block with an infinity or a
// NaN has the scale byte 255, which every reader takes as NaN.
// Products: y = Q(x~) W^T, sums in fp32 on the scaled matrix instructions.
#include "device_util.h"
#include "kq_internal.h"

#include <math.h>

#include <algorithm>

// The rotation's sums are defined as separately rounded fp32 operations (a fused multiply-add
// of the rescale and a butterfly would round differently from the definition).
#pragma clang fp contract(off)

namespace kq {
namespace {

constexpr int QT = 256;          // threads per workgroup
constexpr int MX_GROUP = 128;    // columns per scale dword; rows are padded to whole groups

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__host__ __device__ inline int64_t mx_pad(int64_t n) { return (n + MX_GROUP - 1) / MX_GROUP * MX_GROUP; }

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

struct ProductArgs {
  const uint8_t* xc;       // rows x Kp / 2
  const uint8_t* xs;
  int64_t rows;            // rows of x
  const uint8_t* wc;       // experts x N x Kp / 2
  const uint8_t* ws;
  int64_t N, kp;
  const int32_t* index;    // slot -> row of x, or NULL: the slot itself
  const int32_t* offsets;  // experts + 1 first slots, or NULL: one layer, slots = rows
  int experts;
  int64_t slots;
  void* y;
  int y_bf16;
  int64_t ldy;
};

// Slots [first, last) of expert e, kept inside [0, slots) whatever the offsets hold.
__device__ __forceinline__ void expert_range(const ProductArgs& a, int e, int64_t& first, int64_t& last) {
  if (!a.offsets) { first = 0; last = a.slots; return; }
  const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
  first = lo < 0 ? 0 : lo > a.slots ? a.slots : lo;
  last = hi < first ? first : hi > a.slots ? a.slots : hi;
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// 64 x 64 outputs per workgroup, one 32 x 32 tile per wave, operands straight from memory.
__global__ __launch_bounds__(256) void mx_product_kernel(ProductArgs a) {
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t first, last, tile = blockIdx.y;
  int e = 0;
  for (;; ++e) {
    if (e == a.experts) return;
    expert_range(a, e, first, last);
    const int64_t tiles = (last - first + 63) / 64;
    if (tile < tiles) break;
    tile -= tiles;
  }
  const int64_t m0 = first + tile * 64 + (w >> 1) * 32, n0 = (int64_t)blockIdx.x * 64 + (w & 1) * 32;
  if (m0 >= last || n0 >= a.N) return;
  const int r = l & 31, q = l >> 5;
  const int64_t slot = m0 + r < last ? m0 + r : last - 1;
  int64_t xr = a.index ? (int64_t)a.index[slot] : slot;
  const bool off = xr < 0 || xr >= a.rows;
  if (off) xr = 0;
  const int64_t wr = n0 + r < a.N ? n0 + r : a.N - 1;
  const uint8_t* xp = a.xc + xr * (a.kp / 2) + 16 * q;
  const uint8_t* wp = a.wc + ((int64_t)e * a.N + wr) * (a.kp / 2) + 16 * q;
  const uint8_t* wsc = a.ws + (int64_t)e * a.N * (a.kp / 32);
  f32x16 acc;
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  for (int64_t k = 0; k < a.kp; k += 64) {
    const i32x4 wv = *(const i32x4*)(wp + k / 2);
    i32x4 xv = {0, 0, 0, 0};
    int sx = 0;
    const int sw = wsc[scale_at(wr, k / 32 + q, a.N)];
    if (!off) {
      xv = *(const i32x4*)(xp + k / 2);
      sx = a.xs[scale_at(xr, k / 32 + q, a.rows)];
    }
    const i32x8 xo = {xv[0], xv[1], xv[2], xv[3], 0, 0, 0, 0}, wo = {wv[0], wv[1], wv[2], wv[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xo, wo, acc, 4, 4, 0, sx, 0, sw);
  }
  if (n0 + r >= a.N) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int64_t m = m0 + (j >> 2) * 8 + q * 4 + (j & 3);
    if (m >= last) continue;
    if (a.y_bf16)
      ((uint16_t*)a.y)[m * a.ldy + n0 + r] = to_bf16(acc[j]);
    else
      ((float*)a.y)[m * a.ldy + n0 + r] = acc[j];
  }
}

constexpr int64_t MX_MAX_ROWS = (int64_t)1 << 30, MX_MAX_N = (int64_t)1 << 24;

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

size_t code_bytes(int64_t rows, int64_t n) { return (size_t)rows * (size_t)(mx_pad(n) / 2); }
size_t scale_bytes(int64_t rows, int64_t n) { return (size_t)rows * (size_t)(mx_pad(n) / 32); }

// Checks the source rows and their processing; *block: the Hadamard block.
kq_status check_rows(const char* fn, const void* src, int type, int64_t rows, int64_t n, int64_t ld,
                     int64_t had, int64_t* block) {
  if (type != KQ_F32 && type != KQ_BF16) return fail(KQ_EINVAL, "%s: type %d of the rows", fn, type);
  if (rows < 0 || rows > MX_MAX_ROWS || n < 1 || n > MX_MAX_N)
    return fail(KQ_ESHAPE, "%s: %lld rows of %lld values", fn, (long long)rows, (long long)n);
  if (ld < n) return fail(KQ_ESHAPE, "%s: leading dimension %lld < %lld", fn, (long long)ld, (long long)n);
  if (rows > 0 && !src) return fail(KQ_EINVAL, "%s: NULL rows", fn);
  if ((uintptr_t)src & (type == KQ_F32 ? 3 : 1)) return fail(KQ_EINVAL, "%s: rows not aligned to their type", fn);
  if (had < 0) return fail(KQ_ESHAPE, "%s: negative Hadamard block", fn);
  const int64_t b = had != 0 ? had : (n & -n);
  if (had == 0 && b > 8192)
    return fail(KQ_ENOTIMPL, "%s: the automatic Hadamard block (the largest power of 2 dividing the "
                "width) exceeds 8192; pass a block of at most 8192", fn);
  if (!is_pow2(b) || b > 8192 || n % b != 0)
    return fail(KQ_ESHAPE, "%s: the Hadamard block must be a power of 2 (<= 8192) dividing the width", fn);
  *block = b;
  return KQ_OK;
}

kq_status launch_quantize(const void* src, int type, int64_t rows, int64_t n, int64_t ld, const float* d,
                          const int8_t* sign, int64_t block, uint8_t* codes, uint8_t* scales,
                          uint16_t* values, int64_t ldv, hipStream_t s) {
  if (rows == 0) return KQ_OK;
  QuantArgs a;
  a.src = src; a.rows = rows; a.n = n; a.ld = ld; a.d = d; a.sign = sign;
  a.had = (int)block; a.isb = (float)(1.0 / sqrt((double)block));
  a.codes = codes; a.scales = scales; a.values = values; a.ldv = ldv;
  a.seg = (int)std::max<int64_t>(4096, block);
  const int64_t nseg = ceil_div(mx_pad(n), a.seg);
  if (rows * nseg > 0x7fffffff) return fail(KQ_ESHAPE, "kq_mxfp4: %lld rows of %lld values", (long long)rows, (long long)n);
  const size_t lds = sizeof(float) * (size_t)a.seg;
  if (type == KQ_F32)
    mx_quantize_kernel<float><<<dim3((unsigned)(rows * nseg)), dim3(QT), lds, s>>>(a);
  else
    mx_quantize_kernel<uint16_t><<<dim3((unsigned)(rows * nseg)), dim3(QT), lds, s>>>(a);
  KQ_LAUNCHED("mx_quantize_kernel");
  return KQ_OK;
}

struct XArgs {
  const void* x; int type; int64_t rows, n, ld; const uint8_t* scales;
  const float* d; const int8_t* sign; int64_t had;
};

// Checks and quantises the activations (unless they are quantised already), then the product.
kq_status product(const char* fn, const XArgs& x, ProductArgs p, int y_type, void* ws, size_t ws_bytes,
                  hipStream_t s) {
  int64_t block = 1;
  if (x.type == KQ_MXFP4) {
    if (x.rows < 0 || x.rows > MX_MAX_ROWS || x.n < 1 || x.n > MX_MAX_N)
      return fail(KQ_ESHAPE, "%s: %lld rows of %lld values", fn, (long long)x.rows, (long long)x.n);
    if (x.ld != mx_pad(x.n)) return fail(KQ_ESHAPE, "%s: quantised rows are contiguous: ldx = %lld", fn, (long long)mx_pad(x.n));
    if (x.rows > 0 && (!x.x || !x.scales)) return fail(KQ_EINVAL, "%s: NULL quantised rows or scales", fn);
    if (!aligned16(x.x) || !aligned16(x.scales)) return fail(KQ_EINVAL, "%s: quantised rows must be 16-byte aligned", fn);
    if (x.d || x.sign || (x.had != 1 && x.had != 0)) return fail(KQ_EINVAL, "%s: quantised rows take no rescale, signs or rotation", fn);
  } else {
    KQ_TRY(check_rows(fn, x.x, x.type, x.rows, x.n, x.ld, x.had, &block));
    if (x.scales) return fail(KQ_EINVAL, "%s: scales go with quantised rows only", fn);
  }
  if (y_type != KQ_F32 && y_type != KQ_BF16) return fail(KQ_EINVAL, "%s: output type %d", fn, y_type);
  if (p.N < 1 || p.N > MX_MAX_N) return fail(KQ_ESHAPE, "%s: %lld output channels", fn, (long long)p.N);
  if (p.ldy < p.N) return fail(KQ_ESHAPE, "%s: ldy %lld < %lld", fn, (long long)p.ldy, (long long)p.N);
  if (!p.wc || !p.ws) return fail(KQ_EINVAL, "%s: NULL weights", fn);
  if (!aligned16(p.wc) || !aligned16(p.ws)) return fail(KQ_EINVAL, "%s: weights must be 16-byte aligned", fn);
  if (p.slots > 0 && !p.y) return fail(KQ_EINVAL, "%s: NULL output", fn);
  if ((uintptr_t)p.y & (y_type == KQ_F32 ? 3 : 1)) return fail(KQ_EINVAL, "%s: output not aligned to its type", fn);
  p.kp = mx_pad(x.n);
  p.rows = x.rows;
  p.y_bf16 = y_type == KQ_BF16;
  if (x.type == KQ_MXFP4) {
    p.xc = (const uint8_t*)x.x;
    p.xs = x.scales;
  } else {
    const size_t need = code_bytes(x.rows, x.n) + scale_bytes(x.rows, x.n);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws)))
      return fail(KQ_EWORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    uint8_t* c = (uint8_t*)ws;
    p.xc = c;
    p.xs = c + code_bytes(x.rows, x.n);
  }
  if (p.slots == 0) return KQ_OK;
  if (x.type != KQ_MXFP4)
    KQ_TRY(launch_quantize(x.x, x.type, x.rows, x.n, x.ld, x.d, x.sign, block, (uint8_t*)p.xc,
                           (uint8_t*)p.xs, nullptr, 0, s));
  const int64_t tiles = ceil_div(p.slots, 64) + (p.offsets ? p.experts : 0);
  if (tiles > 65535) return fail(KQ_ESHAPE, "%s: %lld rows", fn, (long long)p.slots);
  mx_product_kernel<<<dim3((unsigned)ceil_div(p.N, 64), (unsigned)tiles), dim3(256), 0, s>>>(p);
  KQ_LAUNCHED("mx_product_kernel");
  return KQ_OK;
}

}  // namespace
}  // namespace kq

extern "C" kq_status kq_mxfp4_quantize(const void* src, int src_type, int64_t rows, int64_t n, int64_t ld,
                                       const float* d, const int8_t* sign, int64_t had, uint8_t* codes,
                                       uint8_t* scales, uint16_t* values_opt, int64_t ldv, void* stream) {
  using namespace kq;
  int64_t block = 1;
  KQ_TRY(check_rows("kq_mxfp4_quantize", src, src_type, rows, n, ld, had, &block));
  if (rows > 0 && (!codes || !scales)) return fail(KQ_EINVAL, "kq_mxfp4_quantize: NULL argument");
  if (!aligned16(codes) || !aligned16(scales))
    return fail(KQ_EINVAL, "kq_mxfp4_quantize: codes and scales must be 16-byte aligned");
  if (values_opt && ldv < n) return fail(KQ_ESHAPE, "kq_mxfp4_quantize: ldv %lld < %lld", (long long)ldv, (long long)n);
  if ((uintptr_t)values_opt & 1) return fail(KQ_EINVAL, "kq_mxfp4_quantize: values not aligned to their type");
  return launch_quantize(src, src_type, rows, n, ld, d, sign, block, codes, scales, values_opt, ldv,
                         as_stream(stream));
}

extern "C" kq_status kq_mxfp4_workspace(int64_t rows, int64_t n, size_t* bytes) {
  using namespace kq;
  if (!bytes) return fail(KQ_EINVAL, "kq_mxfp4_workspace: NULL argument");
  if (rows < 0 || rows > MX_MAX_ROWS || n < 1 || n > MX_MAX_N)
    return fail(KQ_ESHAPE, "kq_mxfp4_workspace: %lld rows of %lld values", (long long)rows, (long long)n);
  *bytes = code_bytes(rows, n) + scale_bytes(rows, n);
  return KQ_OK;
}

extern "C" kq_status kq_mxfp4_linear(const void* x, int x_type, int64_t rows, int64_t in, int64_t ldx,
                                     const uint8_t* x_scales, const float* d, const int8_t* sign,
                                     int64_t had, const uint8_t* w_codes, const uint8_t* w_scales,
                                     int64_t out, void* y, int y_type, int64_t ldy, void* ws,
                                     size_t ws_bytes, void* stream) {
  using namespace kq;
  ProductArgs p{};
  p.wc = w_codes; p.ws = w_scales; p.N = out; p.experts = 1; p.slots = rows; p.y = y; p.ldy = ldy;
  return product("kq_mxfp4_linear", XArgs{x, x_type, rows, in, ldx, x_scales, d, sign, had}, p, y_type, ws,
                 ws_bytes, as_stream(stream));
}

extern "C" kq_status kq_mxfp4_experts(const void* x, int x_type, int64_t rows, int64_t in, int64_t ldx,
                                      const uint8_t* x_scales, const float* d, const int8_t* sign,
                                      int64_t had, const int32_t* index, int64_t slots,
                                      const int32_t* offsets, int experts, const uint8_t* w_codes,
                                      const uint8_t* w_scales, int64_t out, void* y, int y_type,
                                      int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  using namespace kq;
  const char* fn = "kq_mxfp4_experts";
  if (experts < 1 || experts > 4096) return fail(KQ_ESHAPE, "%s: %d experts (1 .. 4096)", fn, experts);
  if (slots < 0 || slots > MX_MAX_ROWS) return fail(KQ_ESHAPE, "%s: %lld slots", fn, (long long)slots);
  if (!offsets) return fail(KQ_EINVAL, "%s: NULL offsets", fn);
  if (((uintptr_t)offsets | (uintptr_t)index) & 3) return fail(KQ_EINVAL, "%s: offsets or index not aligned", fn);
  if (!index && slots > rows)
    return fail(KQ_ESHAPE, "%s: %lld slots of %lld rows need an index", fn, (long long)slots, (long long)rows);
  ProductArgs p{};
  p.wc = w_codes; p.ws = w_scales; p.N = out; p.index = index; p.offsets = offsets; p.experts = experts;
  p.slots = slots; p.y = y; p.ldy = ldy;
  return product(fn, XArgs{x, x_type, rows, in, ldx, x_scales, d, sign, had}, p, y_type, ws, ws_bytes,
                 as_stream(stream));
}
