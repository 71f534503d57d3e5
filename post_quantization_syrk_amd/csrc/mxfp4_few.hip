// Products with layers held in MXFP4 for few rows of activations (decoding), bound by the bytes
// of the layer: every byte of it is read once, straight into the registers that the matrix
// instructions take, and all of a workgroup's loads are in flight before the first is used.
#include "mxfp4_rows.h"
#include "mxfp4_tiles.h"

#include <math.h>

#include <algorithm>

namespace kq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Activations that the kernel quantises itself.
struct RowArgs {
  const void* x;
  int64_t ld, n;
  const float* d;
  const int8_t* sign;
  int had;
  float isb;
};

// Rotates and quantises the tile's rows into LDS: codes [rows][pitch], then scale dwords
// [rows][steps].
template <typename T, int WAVES, bool LONG>
__device__ __forceinline__ void quantize_rows(const ProductArgs& a, const RowArgs& x, const Tile& t, float* lds,
                                              uint8_t* codes, int* scales) {
  const int rows = t.last - t.m0, lane = threadIdx.x & 63;
  auto source = [&](int r) -> const T* {
    const int row = a.index ? a.index[t.m0 + r] : t.m0 + r;
    return row >= 0 && row < a.rows ? (const T*)x.x + row * x.ld : nullptr;
  };
  for (int64_t c0 = 0; c0 < 2 * a.pitch; c0 += SPAN * WAVES) {
    const int64_t c = c0 + 8 * threadIdx.x;
    float f[8], r[8], next[8];
    const T* p = source(0);
    load_columns<T, false>(p, c, p ? x.n : 0, r);
    const bool scaled = x.d || x.sign;
    if (scaled) factors(x.d, x.sign, c, x.n, f);
    for (int k = 0; k < rows; ++k) {
      if (k + 1 < rows) {
        p = source(k + 1);
        load_columns<T, false>(p, c, p ? x.n : 0, next);
      }
      rotate<WAVES, LONG>(r, scaled, f, x.had, x.isb, lds);
      float s;
      bool bad;
      int four;
      const unsigned w = encode(r, s, bad, four);
      if (c < 2 * a.pitch) {
        *(unsigned*)(codes + k * a.pitch + c / 2) = w;
        if ((lane & 15) == 0) scales[k * a.steps + (c >> 7)] = four;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = next[j];
    }
  }
}

// 16 MT rows of y by 16 NT columns per workgroup: its waves take K in equal parts, U steps of 128
// at a time, and add their sums through LDS in wave order.  A lane holds 16 bytes of one row of
// the layer per step: the first operand of the 16 x 16 x 128 instruction; rows of x are the
// second, so a lane's four sums are neighbouring columns of one row of y.
// T: void for quantised activations, else their type, quantised here (MT = 1).
template <int WAVES, int MT, int NT, int U, bool EXPERTS, typename T>
__global__ __launch_bounds__(64 * WAVES) void mx_few_kernel(ProductArgs a, RowArgs x) {
  constexpr bool FUSED = !__is_void(T);
  constexpr int BM = 16 * MT, BN = 16 * NT, LD = BN + 4;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Tile t;
  t.n0 = blockIdx.x * BN;
  if (EXPERTS) {
    if (!search_rows<BM>(a, blockIdx.y, t)) return;
  } else {
    t.e = 0;
    t.m0 = blockIdx.y * BM;
    t.last = (int)a.slots;
  }
  t.last = min(t.last, t.m0 + BM);
  const int per = (a.steps + WAVES - 1) / WAVES, s0 = wave * per, s1 = min(s0 + per, a.steps);

  const uint8_t* wc = a.wc + ((int64_t)t.e * a.N + t.n0) * a.pitch;
  const uint8_t* ws = a.ws + (int64_t)t.e * a.N * (4 * a.steps) + (int64_t)t.n0 * 4;
  unsigned ow[NT], os[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const unsigned r = (unsigned)min((int64_t)16 * n + l16, a.N - 1 - t.n0);
    ow[n] = r * (unsigned)a.pitch + 16 * q;
    os[n] = r * 4;
  }
  // rows of x: quantised ones in memory (zeros for a row outside x), or those quantised below
  const uint8_t* px[MT];
  const uint8_t* ps[MT];
  int64_t stepx[MT], steps[MT];
  const float* spare = lds + rotate_floats(WAVES);
  uint8_t* codes = (uint8_t*)spare;
  int* scales = (int*)(codes + (t.last - t.m0) * a.pitch);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int slot = min(t.m0 + 16 * m + l16, t.last - 1);
    if (FUSED) {
      px[m] = codes + (slot - t.m0) * a.pitch + 16 * q;
      ps[m] = (const uint8_t*)(scales + (slot - t.m0) * a.steps);
      stepx[m] = 64;
      steps[m] = 4;
    } else {
      const int row = EXPERTS && a.index ? a.index[slot] : slot;
      const bool in = row >= 0 && row < a.rows;
      px[m] = in ? a.xc + row * a.pitch + 16 * q : (const uint8_t*)g_zeros;
      ps[m] = in ? a.xs + (int64_t)row * 4 : (const uint8_t*)g_zeros;
      stepx[m] = in ? 64 : 0;
      steps[m] = in ? a.rows * 4 : 0;
    }
  }
  i32x4 wv[U][NT], xv[U][MT];
  int sw[U][NT], sx[U][MT];
  auto load_w = [&](int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = min(s + u, s1 - 1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        wv[u][n] = *(const i32x4*)(wc + 64 * k + ow[n]);
        sw[u][n] = *(const int*)(ws + 4 * a.N * k + os[n]);
      }
    }
  };
  auto load_x = [&](int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = min(s + u, s1 - 1);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        xv[u][m] = *(const i32x4*)(px[m] + stepx[m] * k);
        sx[u][m] = *(const int*)(ps[m] + steps[m] * k);
      }
    }
  };
  if (s0 < s1) load_w(s0);
  if constexpr (FUSED) {
    if (x.had <= SPAN)
      quantize_rows<T, WAVES, false>(a, x, t, lds, codes, scales);
    else
      quantize_rows<T, WAVES, true>(a, x, t, lds, codes, scales);
    __syncthreads();
  }
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{};
  for (int s = s0; s < s1; s += U) {
    if (s > s0) load_w(s);
    load_x(s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              widen(wv[u][n]), widen(xv[u][m]), acc[m][n], 4, 4, 0, sw[u][n] >> (8 * q), 0, sx[u][m] >> (8 * q));
    }
  }
  // sums [wave][row][column]
  if (FUSED) __syncthreads();   // the rotation's buffer has been read
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(f32x4*)(lds + ((wave * BM + 16 * m + l16) * LD + 16 * n + 4 * q)) = acc[m][n];
  __syncthreads();
  const int count = (t.last - t.m0) * BN;
  for (int o = threadIdx.x; o < count; o += 64 * WAVES) {
    const int r = o / BN, c = o % BN;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += lds[(w * BM + r) * LD + c];
    if (t.n0 + c >= a.N) continue;
    const int64_t at = (t.m0 + r) * a.ldy + t.n0 + c;
    if (a.y_bf16)
      ((uint16_t*)a.y)[at] = to_bf16(v);
    else
      ((float*)a.y)[at] = v;
  }
}

template <int WAVES, int MT, int NT, int U, typename T>
kq_status launch(const ProductArgs& p, const RowArgs& x, hipStream_t s) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  const int64_t tm = ceil_div(p.slots, BM) + (p.offsets ? std::min<int64_t>(p.experts, p.slots) : 0);
  size_t bytes = sizeof(float) * (size_t)WAVES * BM * (BN + 4);
  if (!__is_void(T))
    bytes = std::max(bytes, sizeof(float) * (size_t)rotate_floats(WAVES) +
                                (size_t)std::min<int64_t>(p.slots, BM) * (size_t)(p.pitch + 4 * p.steps));
  const dim3 grid((unsigned)ceil_div(p.N, BN), (unsigned)tm), block(64 * WAVES);
  const auto kernel = p.offsets ? mx_few_kernel<WAVES, MT, NT, U, true, T> : mx_few_kernel<WAVES, MT, NT, U, false, T>;
  if (bytes > 64 * 1024)
    KQ_HIP(hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  kernel<<<grid, block, bytes, s>>>(p, x);
  KQ_LAUNCHED("mx_few_kernel");
  return KQ_OK;
}

// Rows of a tile: the fewest that hold the rows per expert, on average, in one.
int few_rows(const ProductArgs& p) {
  const int64_t avg = p.offsets ? ceil_div(p.slots, p.experts) : p.slots;
  return avg <= 16 ? 16 : avg <= 32 ? 32 : 64;
}

}  // namespace

bool mx_few(const ProductArgs& p) {
  const int64_t avg = p.offsets ? ceil_div(p.slots, p.experts) : p.slots;
  return avg <= testing_value(KQ_TESTING_MX_FEW, 64) && p.slots <= 65535 && p.rows * p.pitch < 0x7fffffff;
}

bool mx_few_fused(const ProductArgs& p, const MxRows& x, int64_t block) {
  return p.slots <= 16 && p.slots * x.n <= testing_value(KQ_TESTING_MX_FUSED, 8192) && block <= 8192;
}

kq_status mx_few_product(const ProductArgs& p, const MxRows& x, int64_t block, bool fused, hipStream_t s) {
  RowArgs r{x.x, x.ld, x.n, x.d, x.sign, (int)block, (float)(1.0 / sqrt((double)block))};
  const int bm = fused ? 16 : few_rows(p);
  // waves per workgroup: enough of them to fill the card (eight per SIMD and more), as long as
  // each has two steps of K
  const int64_t tiles = ceil_div(p.N, 16) * (p.offsets ? std::min<int64_t>(p.slots, std::max<int64_t>(p.experts, ceil_div(p.slots, bm)))
                                                       : ceil_div(p.slots, bm));
  const int64_t want = ceil_div(device_cu_count() * 12, tiles);
  int waves = want <= 4 ? 4 : want <= 8 ? 8 : 16;
  while (waves > 4 && p.steps < 2 * waves) waves /= 2;
  if (fused) {
    if (block > 4096) waves = 16;
    else if (block > 2048) waves = std::max(waves, 8);
    const bool f32 = x.type == KQ_F32;
    switch (waves) {
      case 4: return f32 ? launch<4, 1, 1, 8, float>(p, r, s) : launch<4, 1, 1, 8, uint16_t>(p, r, s);
      case 8: return f32 ? launch<8, 1, 1, 8, float>(p, r, s) : launch<8, 1, 1, 8, uint16_t>(p, r, s);
      default: return f32 ? launch<16, 1, 1, 4, float>(p, r, s) : launch<16, 1, 1, 4, uint16_t>(p, r, s);
    }
  }
  if (bm == 16)
    return waves == 4 ? launch<4, 1, 1, 8, void>(p, r, s) : waves == 8 ? launch<8, 1, 1, 8, void>(p, r, s)
                                                                       : launch<16, 1, 1, 4, void>(p, r, s);
  if (bm == 32) return waves == 4 ? launch<4, 2, 2, 4, void>(p, r, s) : launch<8, 2, 2, 4, void>(p, r, s);
  return waves == 4 ? launch<4, 4, 2, 2, void>(p, r, s) : launch<8, 4, 2, 2, void>(p, r, s);
}

}  // namespace kq
