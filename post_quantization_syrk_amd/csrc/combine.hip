// The sum of the experts' rows back to the rows that they came from, and its gradients.
#include "device_util.h"
#include "kq_internal.h"
#include "lanes.h"

#include <algorithm>

namespace kq {
namespace {

constexpr int VEC = 8;   // neighbouring columns of a lane
constexpr int MAX_TOP = 64;

// Eight neighbouring values, read and written 16 bytes at a time at any alignment of their type (as
// single values the compiler takes them apart: 32768 x 2048 x 6 backwards 525 us, so 338).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T>
struct Pack {
  static constexpr int WORDS = VEC * (int)sizeof(T) / 16;
  u32x4 v[WORDS];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(v[i / 4][i % 4]);
    else
      return __uint_as_float(i & 1 ? v[0][i / 2] & 0xffff0000u : v[0][i / 2] << 16);
  }
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ unsigned pair(float lo, float hi) { return __builtin_bit_cast(unsigned, bf16x2{(__bf16)lo, (__bf16)hi}); }
__device__ __forceinline__ void put(float v, float& to) { to = v; }
__device__ __forceinline__ void put(float v, uint16_t& to) { to = __builtin_bit_cast(uint16_t, (__bf16)v); }

// Columns c .. c + 7 of a row of n (zeros past its end).  STREAM: past the caches
// (streams() below).
template <bool STREAM, typename T>
__device__ __forceinline__ Pack<T> load(const T* row, int64_t c, int64_t n) {
  Pack<T> k{};
  if (c + VEC <= n) {
    const u32x4_any* from = (const u32x4_any*)(row + c);
#pragma unroll
    for (int i = 0; i < Pack<T>::WORDS; ++i) k.v[i] = STREAM ? __builtin_nontemporal_load(from + i) : from[i];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i < n) {
        if constexpr (sizeof(T) == 4)
          k.v[i / 4][i % 4] = __float_as_uint(row[c + i]);
        else
          k.v[0][i / 2] |= (unsigned)row[c + i] << (16 * (i & 1));
      }
  }
  return k;
}
template <bool STREAM, typename T>
__device__ __forceinline__ void store(T* row, int64_t c, int64_t n, const float (&v)[VEC]) {
  if (c + VEC <= n) {
    Pack<T> w;
    if constexpr (sizeof(T) == 4) {
      w.v[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      w.v[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      w.v[0] = u32x4{pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])};
    }
    u32x4_any* to = (u32x4_any*)(row + c);
#pragma unroll
    for (int i = 0; i < Pack<T>::WORDS; ++i) {
      if constexpr (STREAM)
        __builtin_nontemporal_store(w.v[i], to + i);
      else
        to[i] = w.v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i < n) put(v[i], row[c + i]);
  }
}

struct CombineArgs {
  const void* z;
  int64_t slots, n, ldz;
  const int32_t* slot;
  const float* weight;
  int64_t rows;
  int top;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  int64_t chunks;   // lanes that share a row
};

// y[t] = residual[t] + sum_j weight[t, j] z[slot[t, j]]: a lane's eight columns of a row, one choice after
// another, sums in registers.  Bound by HBM: 32768 x 2048, top 6, bf16, 183 us, 5.9 TB/s (a large copy:
// 4.9); rows that begin inside a dword, 4099 x 4100, top 2, to fp32: 32 us with its inputs in the last
// cache, 40 without.
template <typename Z, typename Y, typename R, bool STREAM>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t units = a.rows * a.chunks;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int64_t t = u / a.chunks, c = (u - t * a.chunks) * VEC;
    float acc[VEC] = {};
    if (a.residual) {
      const Pack<R> r = load<STREAM>((const R*)a.residual + t * a.ldr, c, a.n);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = r[i];
    }
    for (int j = 0; j < a.top; ++j) {
      const int s = a.slot[t * a.top + j];
      const float w = a.weight ? a.weight[t * a.top + j] : 1.f;
      Pack<Z> k{};
      if (s >= 0 && s < a.slots) k = load<STREAM>((const Z*)a.z + s * a.ldz, c, a.n);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += w * k[i];
    }
    store<STREAM>((Y*)a.y + t * a.ldy, c, a.n, acc);
  }
}

struct BackArgs {
  const void* dy;
  int64_t rows, n, lddy;
  const void* z;
  int64_t slots, ldz;
  const int32_t* slot;
  const float* weight;
  int top;
  void* dz;
  int64_t lddz;
  float* dweight;
};

// dz[slot] = weight dy, dweight = <dy, z[slot]>: a row per workgroup of WAVES, KB choices at a time, whose
// reads go out together, each choice's slot being the same for all lanes; dy is read once for all of
// them.  Bound by HBM: 32768 x 2048, top 6, bf16, 322 us, 5.4 TB/s.  One wave a row up to 1536 columns, which it
// takes in three passes and without a barrier, four above (bf16, top 8: 16384 rows of 1024 121 us, with four
// waves 130, of 1536 173 and 171, of 2048 247 and 229; 64 rows of 2048 10 and 6, of 16384 60 and 20).
template <typename D, typename Z, int WAVES, int KB, bool STREAM>
__global__ __launch_bounds__(64 * WAVES) void combine_backward_kernel(BackArgs a) {
  __shared__ float sums[WAVES][KB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const D* dy = (const D*)a.dy + t * a.lddy;
    for (int j0 = 0; j0 < a.top; j0 += KB) {
      int s[KB];
      float w[KB], dot[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t at = t * a.top + min(j0 + j, a.top - 1);
        const int k = __builtin_amdgcn_readfirstlane(a.slot[at]);
        s[j] = j0 + j < a.top && k >= 0 && k < a.slots ? k : -1;
        w[j] = a.weight ? a.weight[at] : 1.f;
        dot[j] = 0.f;
      }
      for (int64_t c = threadIdx.x * VEC; c < a.n; c += 64 * WAVES * VEC) {
        const Pack<D> d = load<STREAM>(dy, c, a.n);
        Pack<Z> z[KB];
        if (a.dweight) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (s[j] >= 0) z[j] = load<STREAM>((const Z*)a.z + s[j] * a.ldz, c, a.n);
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (s[j] >= 0) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) dot[j] += d[i] * z[j][i];
            }
        }
        if (a.dz) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (s[j] >= 0) {
              float v[VEC];
#pragma unroll
              for (int i = 0; i < VEC; ++i) v[i] = w[j] * d[i];
              store<STREAM>((Z*)a.dz + s[j] * a.lddz, c, a.n, v);
            }
        }
      }
      if (!a.dweight) continue;
#pragma unroll
      for (int j = 0; j < KB; ++j) dot[j] = reduce_lanes<64>(dot[j], [](float x, float y) { return x + y; });
      if constexpr (WAVES > 1) {
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (lane == 0) sums[wave][j] = dot[j];
        __syncthreads();
        if (threadIdx.x < KB && j0 + (int)threadIdx.x < a.top) {
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < WAVES; ++k) v += sums[k][threadIdx.x];
          a.dweight[t * a.top + j0 + threadIdx.x] = v;
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (lane == j && j0 + j < a.top) a.dweight[t * a.top + j0 + j] = dot[j];
      }
    }
  }
}

bool typed(int t) { return t == KQ_F32 || t == KQ_BF16; }
bool off_type(const void* p, int t) { return (uintptr_t)p & (t == KQ_F32 ? 3 : 1); }

constexpr int64_t MAX_ROWS = (int64_t)1 << 30, MAX_N = (int64_t)1 << 24;

// What both directions ask of z's slots, the choices and the rows.
kq_status check_choices(const char* fn, int z_type, int64_t slots, int64_t n, int64_t ldz, const int32_t* slot, const float* weight,
                        int64_t rows, int top) {
  if (!typed(z_type)) return fail(KQ_EINVAL, "%s: z of type %d", fn, z_type);
  if (rows < 0 || rows > MAX_ROWS || slots < 0 || slots > MAX_ROWS || n < 1 || n > MAX_N)
    return fail(KQ_ESHAPE, "%s: %lld rows, %lld slots of %lld values", fn, (long long)rows, (long long)slots, (long long)n);
  if (top < 1 || top > MAX_TOP || rows * top > 0x7fffffff) return fail(KQ_ESHAPE, "%s: top %d (1 .. %d) of %lld rows", fn, top, MAX_TOP, (long long)rows);
  if (ldz < n) return fail(KQ_ESHAPE, "%s: ldz %lld < %lld", fn, (long long)ldz, (long long)n);
  if (rows > 0 && !slot) return fail(KQ_EINVAL, "%s: NULL slot", fn);
  if (((uintptr_t)slot | (uintptr_t)weight) & 3) return fail(KQ_EINVAL, "%s: slot or weight not aligned", fn);
  return KQ_OK;
}

// Whether the rows of z that a call can name are more than the last cache (256 MB) holds: then nothing is kept
// in it, y included.  32768 x 2048, top 6, bf16, 805 MB of z: the sum 190 us, through the caches 211; with a
// pass that reads y after it 233 and 262, and 239 with y alone through the caches; both gradients 353 and 358.
// z of 4096 rows there, 17 MB, each named by 48 choices: 172 us past the caches, 131 through them.  4099 x
// 4100, top 2, 67 MB of z: 40 to 42 us either way.
bool streams(int64_t slots, int64_t rows, int64_t top, int64_t n, size_t size) {
  return std::min(slots, rows * top) * n * (int64_t)size > ((int64_t)256 << 20);
}

template <typename Z, typename Y, typename R>
kq_status launch_combine(const CombineArgs& a, hipStream_t s) {
  const int64_t blocks = std::min(ceil_div(a.rows * a.chunks, 256), MAX_GROUPS);
  const auto kernel = streams(a.slots, a.rows, a.top, a.n, sizeof(Z)) ? combine_kernel<Z, Y, R, true> : combine_kernel<Z, Y, R, false>;
  kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a);
  KQ_LAUNCHED("combine_kernel");
  return KQ_OK;
}

template <typename D, typename Z, int KB>
kq_status launch_backward(const BackArgs& a, hipStream_t s) {
  const bool stream = streams(a.slots, a.rows, a.top, a.n, sizeof(Z)), wide = a.n > 64 * VEC * 3;
  const auto kernel = wide ? (stream ? combine_backward_kernel<D, Z, 4, KB, true> : combine_backward_kernel<D, Z, 4, KB, false>)
                           : (stream ? combine_backward_kernel<D, Z, 1, KB, true> : combine_backward_kernel<D, Z, 1, KB, false>);
  kernel<<<dim3((unsigned)std::min(a.rows, MAX_GROUPS)), dim3(wide ? 256 : 64), 0, s>>>(a);
  KQ_LAUNCHED("combine_backward_kernel");
  return KQ_OK;
}
template <typename D, typename Z>
kq_status launch_backward(const BackArgs& a, hipStream_t s) {
  return a.top <= 2 ? launch_backward<D, Z, 2>(a, s) : a.top <= 4 ? launch_backward<D, Z, 4>(a, s) : launch_backward<D, Z, 8>(a, s);
}

}  // namespace
}  // namespace kq

extern "C" kq_status kq_combine(const void* z, int z_type, int64_t slots, int64_t n, int64_t ldz, const int32_t* slot,
                                const float* weight, int64_t rows, int top, const void* residual, int residual_type,
                                int64_t ldr, void* y, int y_type, int64_t ldy, void* stream) {
  using namespace kq;
  const char* fn = "kq_combine";
  KQ_TRY(check_choices(fn, z_type, slots, n, ldz, slot, weight, rows, top));
  if (!typed(y_type)) return fail(KQ_EINVAL, "%s: y of type %d", fn, y_type);
  if (ldy < n) return fail(KQ_ESHAPE, "%s: ldy %lld < %lld", fn, (long long)ldy, (long long)n);
  if (rows > 0 && !y) return fail(KQ_EINVAL, "%s: NULL y", fn);
  if (rows > 0 && slots > 0 && !z) return fail(KQ_EINVAL, "%s: NULL z", fn);
  if (off_type(z, z_type) || off_type(y, y_type)) return fail(KQ_EINVAL, "%s: z or y not aligned to its type", fn);
  if (residual) {
    if (!typed(residual_type)) return fail(KQ_EINVAL, "%s: residual of type %d", fn, residual_type);
    if (ldr < n) return fail(KQ_ESHAPE, "%s: ldr %lld < %lld", fn, (long long)ldr, (long long)n);
    if (off_type(residual, residual_type)) return fail(KQ_EINVAL, "%s: residual not aligned to its type", fn);
    if (residual == y && rows > 0 && (residual_type != y_type || ldr != ldy)) return fail(KQ_EINVAL, "%s: in place, the residual has y's type and leading dim", fn);
  }
  if (rows == 0) return KQ_OK;
  const CombineArgs a{z, slots, n, ldz, slot, weight, rows, top, residual, ldr, y, ldy, ceil_div(n, VEC)};
  hipStream_t s = as_stream(stream);
#define KQ_COMBINE(Z, Y) \
  (residual_type == KQ_F32 || !residual ? launch_combine<Z, Y, float>(a, s) : launch_combine<Z, Y, uint16_t>(a, s))
  if (z_type == KQ_F32) return y_type == KQ_F32 ? KQ_COMBINE(float, float) : KQ_COMBINE(float, uint16_t);
  return y_type == KQ_F32 ? KQ_COMBINE(uint16_t, float) : KQ_COMBINE(uint16_t, uint16_t);
#undef KQ_COMBINE
}

extern "C" kq_status kq_combine_backward(const void* dy, int dy_type, int64_t rows, int64_t n, int64_t lddy, const void* z,
                                         int z_type, int64_t slots, int64_t ldz, const int32_t* slot, const float* weight,
                                         int top, void* dz_opt, int64_t lddz, float* dweight_opt, void* stream) {
  using namespace kq;
  const char* fn = "kq_combine_backward";
  KQ_TRY(check_choices(fn, z_type, slots, n, ldz, slot, weight, rows, top));
  if (!typed(dy_type)) return fail(KQ_EINVAL, "%s: dy of type %d", fn, dy_type);
  if (lddy < n) return fail(KQ_ESHAPE, "%s: lddy %lld < %lld", fn, (long long)lddy, (long long)n);
  if (rows > 0 && !dy) return fail(KQ_EINVAL, "%s: NULL dy", fn);
  if (rows > 0 && slots > 0 && dweight_opt && !z) return fail(KQ_EINVAL, "%s: NULL z", fn);
  if (dz_opt && lddz < n) return fail(KQ_ESHAPE, "%s: lddz %lld < %lld", fn, (long long)lddz, (long long)n);
  if (off_type(dy, dy_type) || off_type(z, z_type) || off_type(dz_opt, z_type) || ((uintptr_t)dweight_opt & 3))
    return fail(KQ_EINVAL, "%s: an argument is not aligned to its type", fn);
  if (dz_opt && dz_opt == z && lddz != ldz) return fail(KQ_EINVAL, "%s: in place, lddz is ldz", fn);
  if (rows == 0 || (!dz_opt && !dweight_opt)) return KQ_OK;
  const BackArgs a{dy, rows, n, lddy, z, slots, ldz, slot, weight, top, dz_opt, lddz, dweight_opt};
  hipStream_t s = as_stream(stream);
  if (dy_type == KQ_F32) return z_type == KQ_F32 ? launch_backward<float, float>(a, s) : launch_backward<float, uint16_t>(a, s);
  return z_type == KQ_F32 ? launch_backward<uint16_t, float>(a, s) : launch_backward<uint16_t, uint16_t>(a, s);
}
