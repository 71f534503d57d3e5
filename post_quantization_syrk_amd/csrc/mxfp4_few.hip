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
// [rows][steps].  A rotation block takes S waves (LOGH <= 10: one), and the workgroup's waves take
// blocks of the rows one after another.
template <typename T, int WAVES, int LOGH, bool WIDE>
__device__ __forceinline__ void quantize_rows(const ProductArgs& a, const RowArgs& x, const Tile& t, float* lds,
                                              uint8_t* codes, int* scales) {
  constexpr int S = LOGH > 10 ? 1 << (LOGH - 10) : 1, GROUPS = WAVES / S;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int parts = (int)((2 * a.pitch + SPAN * S - 1) / (SPAN * S)), units = parts * (t.last - t.m0);
  const bool scaled = x.d || x.sign, whole = whole_factors(x.d, x.sign, x.n);
  for (int u0 = 0; u0 < units; u0 += GROUPS) {   // every wave passes the barriers of a long block
    const int u = min(u0 + wave / S, units - 1), k = u / parts;
    const int64_t c = (int64_t)(u % parts) * (SPAN * S) + 16 * ((wave % S) * 64 + lane);
    const int row = a.index ? a.index[t.m0 + k] : t.m0 + k;
    const bool in = row >= 0 && row < a.rows;
    Raw<T> raw;
    load_columns<WIDE>((const T*)x.x + (in ? row : 0) * x.ld, c, in ? x.n : 1, raw);
    float r[16], f[16];
    if (scaled) {
      if (whole)
        factors<true>(x.d, x.sign, c, x.n, f);
      else
        factors<false>(x.d, x.sign, c, x.n, f);
    }
    convert<WIDE>(raw, c, x.n, r);
    if (!in) {
#pragma unroll
      for (int j = 0; j < 16; ++j) r[j] = 0.f;
    }
    rotate<WAVES, LOGH>(r, scaled, f, x.had, x.isb, lds);
    float s;
    bool bad;
    int four;
    const u32x2 w = encode<exact_shift(LOGH)>(r, s, bad, four);
    if (c < 2 * a.pitch && u0 + wave / S < units) {
      *(u32x2*)(codes + k * a.pitch + c / 2) = w;
      if ((lane & 7) == 0) scales[k * a.steps + (c >> 7)] = four;
    }
  }
}

// 16 MT rows of y by 16 NT columns per workgroup: its waves take K in equal parts, U pairs of
// 128 at a time, and add their sums through LDS in wave order.  Rows of the layer are the first
// operand of the 16 x 16 x 128 instruction and rows of x the second, so a lane's four sums are
// neighbouring columns of one row of y.  Which 32 of K a lane's operand holds is free as long as
// both operands agree: lane group q takes blocks 2 q and 2 q + 1 of a pair's eight, one per
// instruction, so its two loads are neighbours, a row's line is read whole, and both blocks'
// scales lie in one dword.
// Bound by the layer's bytes and, at these sizes, by the latency of the loads before the first
// product (16 rows, 11008 x 4096: 24 MB, 6.8 us; 2 experts of it for one token: 48 MB, 14.8 us with
// the token's rotation).
// EPI: as for the tiles; a gated layer's pair lies in two neighbouring sums of a lane (one token, 4096 to
// 2 x 11008 with silu: 14.6 us; to 22016 plain: 14.0).
// T: void for quantised activations, else their type, quantised here (MT = 1).
template <int WAVES, int MT, int NT, int U, bool EXPERTS, typename T, bool WIDE, int EPI>
__global__ __launch_bounds__(64 * WAVES, 4) void mx_few_kernel(ProductArgs a, RowArgs x) {
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
  const int pairs = (a.steps + 1) / 2, per = (pairs + WAVES - 1) / WAVES;
  const int p0 = wave * per, p1 = min(p0 + per, pairs);

  const int w0 = first_row<EPI>(t.n0);
  const uint8_t* wc = a.wc + ((int64_t)t.e * a.N + w0) * a.pitch;
  const uint8_t* ws = a.ws + (int64_t)t.e * a.N * (4 * a.steps) + (int64_t)w0 * 4;
  unsigned ow[NT], os[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const unsigned r = (unsigned)layer_row<EPI>(a, t.n0, 16 * n + l16);
    ow[n] = r * (unsigned)a.pitch + 32 * q;
    os[n] = r * 4;
  }
  // rows of x: quantised ones in memory (zeros for a row outside x), or those quantised below
  const uint8_t* px[MT];
  const uint8_t* ps[MT];
  int64_t stepx[MT], steps[MT];
  uint8_t* codes = (uint8_t*)(lds + rotate_floats(WAVES));
  int* scales = (int*)(codes + (t.last - t.m0) * a.pitch);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int slot = min(t.m0 + 16 * m + l16, t.last - 1);
    if (FUSED) {
      px[m] = codes + (slot - t.m0) * a.pitch + 32 * q;
      ps[m] = (const uint8_t*)(scales + (slot - t.m0) * a.steps);
      stepx[m] = 64;
      steps[m] = 4;
    } else {
      const int row = EXPERTS && a.index ? a.index[slot] : slot;
      const bool in = row >= 0 && row < a.rows;
      px[m] = in ? a.xc + row * a.pitch + 32 * q : (const uint8_t*)g_zeros;
      ps[m] = in ? a.xs + (int64_t)row * 4 : (const uint8_t*)g_zeros;
      stepx[m] = in ? 64 : 0;
      steps[m] = in ? a.rows * 4 : 0;
    }
  }
  // Pair p of the lane: its first step of 128 is 2 p + q / 2.  The last pair may lack its second
  // step: lane groups 2 and 3 then read the first one's again and take zeros for x.
  i32x4 wv[U][NT][2], xv[U][MT][2];
  int sw[U][NT], sx[U][MT];
  auto lacks = [&](int p) { return 2 * p + 1 >= a.steps && q >= 2; };
  auto load_w = [&](int first) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = min(first + u, p1 - 1), back = lacks(p);
      const int64_t k = 2 * p + (q >> 1) - back;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint8_t* from = wc + 128 * (int64_t)p + (ow[n] - 64 * back);
        wv[u][n][0] = *(const i32x4*)from;
        wv[u][n][1] = *(const i32x4*)(from + 16);
        sw[u][n] = *(const int*)(ws + 4 * a.N * k + os[n]);
      }
    }
  };
  auto load_x = [&](int first) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = min(first + u, p1 - 1), back = lacks(p);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint8_t* from = px[m] + stepx[m] * (2 * p - back);
        xv[u][m][0] = *(const i32x4*)from;
        xv[u][m][1] = *(const i32x4*)(from + (stepx[m] >> 2));
        sx[u][m] = *(const int*)(ps[m] + steps[m] * (2 * p + (q >> 1) - back));
        if (2 * p + 1 >= a.steps) {
          xv[u][m][0] = back ? i32x4{} : xv[u][m][0];
          xv[u][m][1] = back ? i32x4{} : xv[u][m][1];
        }
      }
    }
  };
  if (p0 < p1) load_w(p0);
  if constexpr (FUSED) {
    switch (x.had > SPAN ? x.had / SPAN : 1) {
      case 2: quantize_rows<T, WAVES, 11, WIDE>(a, x, t, lds, codes, scales); break;
      case 4: quantize_rows<T, WAVES, 12, WIDE>(a, x, t, lds, codes, scales); break;
      case 8: quantize_rows<T, WAVES, 13, WIDE>(a, x, t, lds, codes, scales); break;
      default: quantize_rows<T, WAVES, -1, WIDE>(a, x, t, lds, codes, scales); break;
    }
    __syncthreads();
  }
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{};
  const int shift = 16 * (q & 1);   // the lane's two scales: bytes 2 q and 2 q + 1 of a pair's eight
  for (int p = p0; p < p1; p += U) {
    if (p > p0) load_w(p);
    load_x(p);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p + u >= p1) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int s = sw[u][n] >> shift, v = sx[u][m] >> shift;
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(wv[u][n][0]), widen(xv[u][m][0]),
                                                                       acc[m][n], 4, 4, 0, s, 0, v);
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(wv[u][n][1]), widen(xv[u][m][1]),
                                                                       acc[m][n], 4, 4, 1, s, 1, v);
        }
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
  constexpr int PAIR = EPI == EPI_GATED ? 2 : 1, COLS = BN / PAIR;
  const int count = (t.last - t.m0) * COLS;
  for (int o = threadIdx.x; o < count; o += 64 * WAVES) {
    const int r = o / COLS, c = o % COLS;
    float v = 0.f, u = 0.f;   // (gated: a pair, in one read)
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float* from = lds + (w * BM + r) * LD + PAIR * c;
      if constexpr (EPI == EPI_GATED) {
        const float2 both = *(const float2*)from;
        v += both.x;
        u += both.y;
      } else {
        v += *from;
      }
    }
    if (t.n0 + PAIR * c >= a.N) continue;
    if constexpr (EPI != EPI_NONE) {
      const float* bias = a.bias + (int64_t)t.e * a.N + w0 + c;
      if (a.bias) v += *bias;
      float half[1] = {v};
      activate(a.act, half);
      v = half[0];
      if constexpr (EPI == EPI_GATED) {
        if (a.bias) u += bias[a.N >> 1];
        v *= u;
      }
      if (a.residual) {
        const int64_t from = (t.m0 + r) * a.ldr + w0 + c;
        v += a.r_bf16 ? __uint_as_float((unsigned)((const uint16_t*)a.residual)[from] << 16) : ((const float*)a.residual)[from];
      }
    }
    const int64_t at = (t.m0 + r) * a.ldy + w0 + c;
    if (a.y_bf16)
      ((uint16_t*)a.y)[at] = to_bf16(v);
    else
      ((float*)a.y)[at] = v;
  }
}

template <int WAVES, int MT, int NT, int U, typename T, bool WIDE, int EPI>
kq_status launch_epi(const ProductArgs& p, const RowArgs& x, hipStream_t s) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  const int64_t tm = ceil_div(p.slots, BM) + (p.offsets ? std::min<int64_t>(p.experts, p.slots) : 0);
  size_t bytes = sizeof(float) * (size_t)WAVES * BM * (BN + 4);
  if (!__is_void(T))
    bytes = std::max(bytes, sizeof(float) * (size_t)rotate_floats(WAVES) +
                                (size_t)std::min<int64_t>(p.slots, BM) * (size_t)(p.pitch + 4 * p.steps));
  const dim3 grid((unsigned)ceil_div(p.N, BN), (unsigned)tm), block(64 * WAVES);
  const auto kernel = p.offsets ? mx_few_kernel<WAVES, MT, NT, U, true, T, WIDE, EPI> : mx_few_kernel<WAVES, MT, NT, U, false, T, WIDE, EPI>;
  if (bytes > 64 * 1024)
    KQ_HIP(hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  kernel<<<grid, block, bytes, s>>>(p, x);
  KQ_LAUNCHED("mx_few_kernel");
  return KQ_OK;
}

template <int WAVES, int MT, int NT, int U, typename T, bool WIDE = true>
kq_status launch(const ProductArgs& p, const RowArgs& x, hipStream_t s) {
  switch (p.epi) {
    case EPI_GATED: return launch_epi<WAVES, MT, NT, U, T, WIDE, EPI_GATED>(p, x, s);
    case EPI_PLAIN: return launch_epi<WAVES, MT, NT, U, T, WIDE, EPI_PLAIN>(p, x, s);
    default: return launch_epi<WAVES, MT, NT, U, T, WIDE, EPI_NONE>(p, x, s);
  }
}

// Rows per expert, on average.
int64_t average_rows(const ProductArgs& p) { return p.offsets ? ceil_div(p.slots, p.experts) : p.slots; }

// Row tiles of bm rows, for rows spread evenly over the experts.
int64_t even_tiles(const ProductArgs& p, int bm) {
  return p.offsets ? std::max<int64_t>(std::min<int64_t>(p.slots, p.experts), ceil_div(p.slots, bm)) : ceil_div(p.slots, bm);
}

}  // namespace

// Where 64 x 64 tiles would leave three compute units of four idle; up to 32 rows where half of
// them; up to 16 where any (64 rows, 4096 x 4096: 6.2 us here, 7.2 in tiles; 256 rows, 1024 x 4096: 6.2
// and 7.2, 384 rows: 8.3 and 7.3; 512 rows, 256 x 9472: 9.9 and 12.3; 32 rows, 4096 x 4096: 5.0 and 7.2,
// 11008 x 4096: 8.7 and 7.4; 16 rows, 11008 x 4096: 7.3 and 7.3; 28672 x 8192: 21.8 and 20.3).
bool mx_few(const ProductArgs& p) {
  const int64_t avg = average_rows(p), tiles = even_tiles(p, 64) * ceil_div(p.N, 64), cus = device_cu_count();
  const int64_t rows = 4 * tiles <= cus ? 65535 : 2 * tiles < cus ? 32 : tiles < cus ? 16 : 0;
  return avg <= testing_value(KQ_TESTING_MX_FEW, rows) && p.slots <= 65535 && p.rows * p.pitch < 0x7fffffff;
}

// One token or two: each workgroup quantises them for itself, while its part of the layer is on
// the way (one token, 4096 x 4096: 7.5 us, and by a kernel of its own 8.2; through two of eight experts of
// 11008 x 4096: 14.8 and 17.7; 6 experts of 4096 x 1024 10.2 and 12.2; but 16 rows, 28672 x 512: 14.1 and 10.2).
bool mx_few_fused(const ProductArgs& p, const MxRows& x) {
  return x.rows > 0 && p.slots <= 16 && p.slots * x.n <= testing_value(KQ_TESTING_MX_FUSED, 8192);
}

kq_status mx_few_product(const ProductArgs& p, const MxRows& x, int64_t block, bool fused, hipStream_t s) {
  RowArgs r{x.x, x.ld, x.n, x.d, x.sign, (int)block, (float)(1.0 / sqrt((double)block))};
  const int bm = fused || average_rows(p) <= 16 ? 16 : 32;
  // Columns per workgroup, 16 to 64: more of them serve its rows of x and its fixed costs, which are worth
  // about 16 columns, and 48 where it quantises the rows too; and what the busiest compute unit has to do
  // counts (16 rows, 4096 x 4096: 3.7 us with 16, 6.5 with 64; 28672 x 8192: 30 and 24; 6 experts of 4096 x 1024
  // for a token each, quantised here: 11.9, with 32 9.0, with 64 7.0).
  const int64_t tm = even_tiles(p, bm), cus = device_cu_count(), fixed = fused ? 48 : 16;
  int nt = 1;
  int64_t least = 0;
  for (int k = bm == 32 ? 2 : 4; k > 0; --k) {
    const int64_t cost = ceil_div(ceil_div(p.N, 16 * k) * tm, cus) * (16 * k + fixed);
    if (least == 0 || cost < least) {
      least = cost;
      nt = k;
    }
  }
  if (fused) {
    const bool f32 = x.type == KQ_F32, wide = wide_rows(x);
#define KQ_FEW(NT, U)                                                                               \
  (f32 ? launch<8, 1, NT, U, float, true>(p, r, s)                                                   \
       : wide ? launch<8, 1, NT, U, uint16_t, true>(p, r, s) : launch<8, 1, NT, U, uint16_t, false>(p, r, s))
    return nt == 4 ? KQ_FEW(4, 1) : nt == 3 ? KQ_FEW(3, 1) : nt == 2 ? KQ_FEW(2, 2) : KQ_FEW(1, 2);
#undef KQ_FEW
  }
  if (bm == 32) return nt == 1 ? launch<8, 2, 1, 2, void>(p, r, s) : launch<8, 2, 2, 2, void>(p, r, s);
  if (nt == 3) return launch<8, 1, 3, 1, void>(p, r, s);
  return nt == 4 ? launch<8, 1, 4, 1, void>(p, r, s) : nt == 2 ? launch<8, 1, 2, 2, void>(p, r, s) : launch<8, 1, 1, 2, void>(p, r, s);
}

}  // namespace kq
