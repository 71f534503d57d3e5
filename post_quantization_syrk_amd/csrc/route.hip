// Routing of rows to a mixture's experts: softmax, the `top` largest logits, slots sorted by expert,
// counts and the balance loss, and the gradient of the logits.
//
// Rows are dealt to waves in contiguous chunks.  A first kernel takes the softmax and the choices of
// its chunks' rows and counts each chunk's choices per expert; a second sums the counts over the
// chunks, which gives every chunk its first slot at each expert; a third gives the chunk's choices
// their slots, in order.  Every order is that of the rows, so nothing depends on timing.
#include "device_util.h"
#include "kq_internal.h"

#include <algorithm>

namespace kq {
namespace {

constexpr int MAX_TOP = 16, MAX_EXPERTS = 4096;
constexpr int WAVES = 4;   // per workgroup of the first and third kernel

struct RouteArgs {
  const void* logits;
  int64_t rows, ld;
  int experts, top;
  bool normalize, wide;   // wide: rows that may be read four values at a time
  float* weight;
  int32_t* expert;
  int32_t* slot;
  int32_t* index;
  int32_t* offsets;
  int32_t* counts;
  float* loss;
  int chunks;
  int64_t per;            // rows of a chunk
  int32_t* hist;          // [chunks][experts + 1]: choices per expert, rows with a softmax
  float* prob;            // [chunks][experts]: sums of probabilities
  double* mean;           // [experts]: over all chunks
};

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((unsigned)v << 16); }

// exp(x) for x <= 0, infinities and NaN among them, to about an ulp: 2^(x log2 e) with what the
// product loses put back.  Below -120 the result is zero in fp32 anyway (and -inf would give NaN).
__device__ __forceinline__ float exp_of(float x) {
  const float c = x < -120.f ? -120.f : x;
  const float t = c * 1.44269502f, r = fmaf(c, 1.44269502f, -t) + c * 1.92596303e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.693147182f, e);
}

// A row's values in registers: LPR lanes hold VPL each, in groups of W = min(VPL, 4) neighbours.
// Value v of lane l is column (v / W) LPR W + l W + v % W, so columns ascend with v in a lane.
template <int LPR, int VPL>
struct Row {
  static constexpr int W = VPL < 4 ? VPL : 4;
  __device__ static constexpr int column(int v) { return v / W * (LPR * W) + v % W; }   // plus W l
};

template <typename T, int LPR, int VPL>
__device__ __forceinline__ void load_row(const T* p, int l, int n, bool wide, float (&r)[VPL]) {
  using R = Row<LPR, VPL>;
  if (wide) {
#pragma unroll
    for (int g = 0; g < VPL / R::W; ++g) {
      const int c = R::column(g * R::W) + R::W * l;
      if constexpr (sizeof(T) == 4) {
        struct __attribute__((packed, aligned(4))) Pack { float v[R::W]; };
        Pack k{};
        if (c < n) k = *(const Pack*)(p + c);
#pragma unroll
        for (int i = 0; i < R::W; ++i) r[g * R::W + i] = c < n ? k.v[i] : -INFINITY;
      } else {
        struct __attribute__((packed, aligned(2))) Pack { uint16_t v[R::W]; };
        Pack k{};
        if (c < n) k = *(const Pack*)(p + c);
#pragma unroll
        for (int i = 0; i < R::W; ++i) r[g * R::W + i] = c < n ? bf16_value(k.v[i]) : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = R::column(v) + R::W * l;
      r[v] = -INFINITY;
      if (c < n) r[v] = sizeof(T) == 4 ? ((const float*)p)[c] : bf16_value(((const uint16_t*)p)[c]);
    }
  }
}

// Over the LPR lanes of a row, the result in all of them.
template <int LPR, typename V, typename F>
__device__ __forceinline__ V reduce_row(V v, F f) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v = f(v, __shfl_xor(v, o));
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  return reduce_row<LPR>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return reduce_row<LPR>(v, [](float a, float b) { return a + b; });
}
template <int LPR>
__device__ __forceinline__ int row_min(int v) {
  return reduce_row<LPR>(v, [](int a, int b) { return min(a, b); });
}

// The rows [r0, r1) of a chunk, by one wave: weights, experts; its choices per expert added to
// hist (LDS, [experts], zero before), its probabilities summed in prob.  Returns its rows with a
// logit above -inf.
template <typename T, int LPR, int VPL>
__device__ __forceinline__ int route_chunk(const RouteArgs& a, int64_t r0, int64_t r1, int* hist, float (&prob)[VPL]) {
  using R = Row<LPR, VPL>;
  constexpr int ROWS = 64 / LPR;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  int used = 0;
  for (int64_t t = r0; t < r1; t += ROWS) {
    const int64_t row = t + lane / LPR;
    const bool in = row < r1;
    float x[VPL];
    load_row<T, LPR, VPL>((const T*)a.logits + (in ? row : r0) * a.ld, l, a.experts, a.wide, x);
    float m = x[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) m = fmaxf(m, x[v]);
    m = row_max<LPR>(m);
    const bool some = m > -INFINITY;   // (of NaN alone: none; its exponentials below are NaN all the same)
    const float base = some ? m : 0.f;
    float p[VPL], sum = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      p[v] = exp_of(x[v] - base);
      sum += p[v];
    }
    sum = row_sum<LPR>(sum);
    const bool bad = !(sum == sum);
    if (a.loss && in) {
      const float inv = some || bad ? 1.f / sum : 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) prob[v] += p[v] * inv;
    }
    used += __popcll(__ballot(in && l == 0 && (some || bad)));
    // one choice after another: the first column of the largest value left
    float total = 0.f, mine = 0.f;
    int chosen = -1;
    for (int j = 0; j < a.top; ++j) {
      float best = x[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) best = fmaxf(best, x[v]);
      best = row_max<LPR>(best);
      int c = 0x7fffffff;
#pragma unroll
      for (int v = VPL - 1; v >= 0; --v) c = x[v] == best ? R::column(v) + R::W * l : c;
      c = row_min<LPR>(c);
      const int own = c - R::W * l;
#pragma unroll
      for (int v = 0; v < VPL; ++v) x[v] = own == R::column(v) ? -INFINITY : x[v];
      const bool there = best > -INFINITY && !bad;
      const float e = there ? exp_of(best - base) : 0.f;
      total += e;
      if (l == j) {
        chosen = there ? c : -1;
        mine = e;
      }
    }
    if (in && l < a.top) {
      const float by = a.normalize ? total : sum;
      a.weight[row * a.top + l] = bad ? NAN : chosen >= 0 ? mine / by : 0.f;
      a.expert[row * a.top + l] = chosen;
      if (chosen >= 0) atomicAdd(hist + chosen, 1);
    }
  }
  return used;
}

// Adds the waves' sums of probabilities, in order, into sums (LDS, [experts], zero before).
template <int LPR, int VPL>
__device__ __forceinline__ void add_prob(const RouteArgs& a, const float (&prob)[VPL], float* sums) {
  using R = Row<LPR, VPL>;
  const int lane = threadIdx.x & 63, l = lane % LPR;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float s = prob[v];
#pragma unroll
    for (int o = LPR; o < 64; o <<= 1) s += __shfl_xor(s, o);
    const int c = R::column(v) + R::W * l;
    if (lane < LPR && c < a.experts) sums[c] = s;
  }
}

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(64 * WAVES) void route_rows_kernel(RouteArgs a) {
  extern __shared__ int lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunk = blockIdx.x * WAVES + wave;
  int* hist = lds + wave * a.experts;
  for (int e = lane; e < a.experts; e += 64) hist[e] = 0;
  __syncthreads();
  if (chunk >= a.chunks) return;
  const int64_t r0 = chunk * a.per, r1 = min(r0 + a.per, a.rows);
  float prob[VPL] = {};
  const int used = route_chunk<T, LPR, VPL>(a, r0, r1, hist, prob);
  int32_t* to = a.hist + (int64_t)chunk * (a.experts + 1);
  for (int e = lane; e < a.experts; e += 64) to[e] = hist[e];
  if (lane == 0) to[a.experts] = used;
  if (a.loss) add_prob<LPR, VPL>(a, prob, a.prob + (int64_t)chunk * a.experts);
}

// Sixteen experts (and, past the last, the count of rows) per workgroup: the chunks' counts become
// the choices of the chunks before, the totals go to counts, the probabilities' sums to mean.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteArgs a) {
  __shared__ int seg[64][17];
  __shared__ double seg_p[64][17];
  const int k = threadIdx.x & 15, s = threadIdx.x >> 4, e = blockIdx.x * 16 + k;
  const int per = (a.chunks + 63) / 64, c0 = min(s * per, a.chunks), c1 = min(c0 + per, a.chunks);
  const int64_t pitch = a.experts + 1;
  int n = 0;
  double p = 0;
  if (e <= a.experts)
    for (int c = c0; c < c1; ++c) n += a.hist[c * pitch + e];
  if (e < a.experts && a.loss)
    for (int c = c0; c < c1; ++c) p += a.prob[(int64_t)c * a.experts + e];
  seg[s][k] = n;
  seg_p[s][k] = p;
  __syncthreads();
  if (e > a.experts) return;
  int before = 0, total = 0;
  for (int i = 0; i < 64; ++i) {
    if (i == s) before = total;
    total += seg[i][k];
  }
  if (s == 0) {
    a.counts[e == a.experts ? e + 1 : e] = total;
    if (e < a.experts && a.loss) {
      double sum = 0;
      for (int i = 0; i < 64; ++i) sum += seg_p[i][k];
      a.mean[e] = sum;
    }
  }
  if (e < a.experts)
    for (int c = c0; c < c1; ++c) {
      const int v = a.hist[c * pitch + e];
      a.hist[c * pitch + e] = before;
      before += v;
    }
}

// Exclusive prefix sums of counts[0 .. n) into first[0 .. n], by one wave.
__device__ __forceinline__ void first_slots(const int32_t* counts, int n, int* first) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int c = e0 + lane < n ? counts[e0 + lane] : 0;
    int sum = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o);
      if (lane >= o) sum += v;
    }
    if (e0 + lane < n) first[e0 + lane] = base + sum - c;
    base += __shfl(sum, 63);
  }
  if (lane == 0) first[n] = base;
}

// Slots for the choices [i0, i1) of a chunk, in order: next[e] (LDS) is the next slot at expert e.
__device__ __forceinline__ void place(const RouteArgs& a, int64_t i0, int64_t i1, int* next) {
  const int lane = threadIdx.x & 63;
  const int bits = 32 - __builtin_clz(a.experts);   // of experts 0 .. experts (none: experts)
  for (int64_t i = i0; i < i1; i += 64) {
    const bool in = i + lane < i1;
    const int e = in ? a.expert[i + lane] : -1;
    const int key = e < 0 ? a.experts : e;
    unsigned long long same = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long set = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int slot = -1;
    if (e >= 0) {
      slot = next[e] + rank;
      if (rank == 0) next[e] = slot + __popcll(same);   // (reads of this round come before: one wave)
    }
    if (in) {
      a.slot[i + lane] = slot;
      if (slot >= 0) a.index[slot] = (int32_t)((i + lane) / a.top);
    }
  }
}

// Offsets, the total, the loss and the index past the last slot, from the counts: one workgroup of
// THREADS; first: the experts' first slots.
template <int THREADS>
__device__ __forceinline__ void finish(const RouteArgs& a, const int* first, double* shared) {
  const int made = first[a.experts];
  for (int e = threadIdx.x; e <= a.experts; e += THREADS) a.offsets[e] = first[e];
  if (threadIdx.x == 0) a.counts[a.experts] = made;
  if (a.loss) {
    const int used = a.counts[a.experts + 1];
    double s = 0;
    for (int e = threadIdx.x; e < a.experts; e += THREADS) s += (double)(first[e + 1] - first[e]) * a.mean[e];
    // (an expert without choices adds nothing, but a NaN probability has to show)
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      s = 0;
      for (int i = 0; i < THREADS / 64; ++i) s += shared[i];
      *a.loss = (float)(s * a.experts / ((double)max(made, 1) * max(used, 1)));
    }
  }
}

__global__ __launch_bounds__(64 * WAVES) void route_place_kernel(RouteArgs a) {
  extern __shared__ int lds[];   // first slots [experts + 1], then each wave's next slots [experts]
  __shared__ double shared[WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave == 0) first_slots(a.counts, a.experts, lds);
  __syncthreads();
  const int made = lds[a.experts];
  for (int64_t i = made + (int64_t)blockIdx.x * (64 * WAVES) + threadIdx.x; i < a.rows * a.top; i += (int64_t)gridDim.x * (64 * WAVES))
    a.index[i] = -1;
  if (blockIdx.x == 0) finish<64 * WAVES>(a, lds, shared);
  const int chunk = blockIdx.x * WAVES + wave;
  if (chunk >= a.chunks) return;
  int* next = lds + a.experts + 1 + wave * a.experts;
  const int32_t* before = a.hist + (int64_t)chunk * (a.experts + 1);
  for (int e = lane; e < a.experts; e += 64) next[e] = lds[e] + before[e];
  const int64_t r0 = chunk * a.per, r1 = min(r0 + a.per, a.rows);
  place(a, r0 * a.top, r1 * a.top, next);
}

struct BackArgs {
  const void* logits;
  int64_t rows, ld, ldd;
  int experts, top;
  bool normalize, wide;
  const float* weight;
  const int32_t* expert;
  const int32_t* counts;
  const float* dweight;
  const float* dloss;
  void* dlogits;
  int64_t per;
};

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(64 * WAVES) void route_backward_kernel(BackArgs a) {
  using R = Row<LPR, VPL>;
  constexpr int ROWS = 64 / LPR;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  const int64_t chunk = blockIdx.x * WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r0 = chunk * a.per, r1 = min(r0 + a.per, a.rows);
  float b[VPL];
  const float unit = a.dloss ? *a.dloss * (float)a.experts / ((float)max(a.counts[a.experts], 1) * (float)max(a.counts[a.experts + 1], 1)) : 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = R::column(v) + R::W * l;
    b[v] = c < a.experts && a.dloss ? unit * (float)a.counts[c] : 0.f;
  }
  for (int64_t t = r0; t < r1; t += ROWS) {
    const int64_t row = t + lane / LPR;
    const bool in = row < r1;
    const int64_t from = in ? row : r0;
    float x[VPL];
    load_row<T, LPR, VPL>((const T*)a.logits + from * a.ld, l, a.experts, a.wide, x);
    int chosen = -1;
    float w = 0.f, g = 0.f;
    if (l < a.top) {
      chosen = a.expert[from * a.top + l];
      if (chosen >= 0 && a.dweight) {
        w = a.weight[from * a.top + l];
        g = a.dweight[from * a.top + l];
      }
    }
    // the softmax once more: a saved logarithm of its sum would be off by 2^-24 of itself, which is
    // the relative error of every exponential
    float m = x[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) m = fmaxf(m, x[v]);
    m = row_max<LPR>(m);
    const float base = m > -INFINITY ? m : 0.f;
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      x[v] = exp_of(x[v] - base);
      sum += x[v];
    }
    sum = row_sum<LPR>(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;   // (no logit above -inf: every p is 0)
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      x[v] *= inv;
      dot += x[v] * b[v];
    }
    dot = row_sum<LPR>(dot);
    const float wg = row_sum<LPR>(w * g);
    const float back = a.normalize ? dot : dot + wg;
    const float extra = a.normalize ? w * (g - wg) : w * g;
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] *= b[v] - back;
    for (int j = 0; j < a.top; ++j) {
      const int own = __shfl(chosen, lane / LPR * LPR + j) - R::W * l;
      const float add = __shfl(extra, lane / LPR * LPR + j);
#pragma unroll
      for (int v = 0; v < VPL; ++v) x[v] += own == R::column(v) ? add : 0.f;
    }
    if (!in) continue;
    T* to = (T*)a.dlogits + row * a.ldd;
#pragma unroll
    for (int g4 = 0; g4 < VPL / R::W; ++g4) {
      const int c = R::column(g4 * R::W) + R::W * l;
      if (a.wide) {
        struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[R::W]; };
        Pack k;
#pragma unroll
        for (int i = 0; i < R::W; ++i) {
          if constexpr (sizeof(T) == 4) k.v[i] = x[g4 * R::W + i];
          else k.v[i] = __builtin_bit_cast(uint16_t, (__bf16)x[g4 * R::W + i]);
        }
        if (c < a.experts) *(Pack*)(to + c) = k;
      } else {
#pragma unroll
        for (int i = 0; i < R::W; ++i)
          if (c + i < a.experts) {
            if constexpr (sizeof(T) == 4) to[c + i] = x[g4 * R::W + i];
            else to[c + i] = __builtin_bit_cast(uint16_t, (__bf16)x[g4 * R::W + i]);
          }
      }
    }
  }
}

// How many chunks the rows are dealt to: four row groups each at least, and as many as the card holds.
void deal(int64_t rows, int experts, int* chunks, int64_t* per) {
  const int64_t most = std::max<int64_t>(512, std::min<int64_t>(2048, (1 << 20) / (experts + 1)));
  *per = std::max<int64_t>(ceil_div(ceil_div(rows, most), 4) * 4, 16);
  *chunks = (int)ceil_div(rows, *per);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

kq_status check_route(const char* fn, const void* logits, int type, int64_t rows, int experts, int64_t ld, int top, int normalize) {
  if (type != KQ_F32 && type != KQ_BF16) return fail(KQ_EINVAL, "%s: logits of type %d", fn, type);
  if (normalize != 0 && normalize != 1) return fail(KQ_EINVAL, "%s: normalize %d", fn, normalize);
  if (experts < 1 || experts > MAX_EXPERTS) return fail(KQ_ESHAPE, "%s: %d experts (1 .. %d)", fn, experts, MAX_EXPERTS);
  if (top < 1 || top > std::min(experts, MAX_TOP)) return fail(KQ_ESHAPE, "%s: top %d of %d experts (at most %d)", fn, top, experts, MAX_TOP);
  if (rows < 0 || rows * (int64_t)top > 0x7fffffff || rows > 0x7fffffff) return fail(KQ_ESHAPE, "%s: %lld rows", fn, (long long)rows);
  if (ld < experts) return fail(KQ_ESHAPE, "%s: ld %lld < %d", fn, (long long)ld, experts);
  if (rows > 0 && !logits) return fail(KQ_EINVAL, "%s: NULL logits", fn);
  if ((uintptr_t)logits & (type == KQ_F32 ? 3 : 1)) return fail(KQ_EINVAL, "%s: logits not aligned to their type", fn);
  return KQ_OK;
}

template <template <typename, int, int> class F, typename A>
kq_status by_width(int type, int experts, const A& a) {
#define KQ_ROUTE(LPR, VPL) (type == KQ_F32 ? F<float, LPR, VPL>::go(a) : F<uint16_t, LPR, VPL>::go(a))
  if (experts <= 16) return KQ_ROUTE(16, 1);
  if (experts <= 32) return KQ_ROUTE(16, 2);
  if (experts <= 64) return KQ_ROUTE(16, 4);
  if (experts <= 128) return KQ_ROUTE(16, 8);
  if (experts <= 256) return KQ_ROUTE(16, 16);
  if (experts <= 512) return KQ_ROUTE(64, 8);
  if (experts <= 1024) return KQ_ROUTE(64, 16);
  if (experts <= 2048) return KQ_ROUTE(64, 32);
  return KQ_ROUTE(64, 64);
#undef KQ_ROUTE
}

struct RouteLaunch {
  RouteArgs a;
  hipStream_t s;
};
template <typename T, int LPR, int VPL>
struct RouteRows {
  static kq_status go(const RouteLaunch& r) {
    RouteArgs a = r.a;
    a.wide = a.experts % Row<LPR, VPL>::W == 0;
    const unsigned grid = (unsigned)ceil_div(a.chunks, WAVES);
    route_rows_kernel<T, LPR, VPL><<<dim3(grid), dim3(64 * WAVES), sizeof(int) * WAVES * (size_t)a.experts, r.s>>>(a);
    KQ_LAUNCHED("route_rows_kernel");
    return KQ_OK;
  }
};

struct BackLaunch {
  BackArgs a;
  hipStream_t s;
};
template <typename T, int LPR, int VPL>
struct RouteBack {
  static kq_status go(const BackLaunch& r) {
    BackArgs a = r.a;
    a.wide = a.experts % Row<LPR, VPL>::W == 0;
    const int64_t units = ceil_div(a.rows, 64 / LPR), waves = std::min<int64_t>(units, (int64_t)device_cu_count() * 32);
    a.per = ceil_div(units, waves) * (64 / LPR);
    const unsigned grid = (unsigned)ceil_div(ceil_div(a.rows, a.per), WAVES);
    route_backward_kernel<T, LPR, VPL><<<dim3(grid), dim3(64 * WAVES), 0, r.s>>>(a);
    KQ_LAUNCHED("route_backward_kernel");
    return KQ_OK;
  }
};

}  // namespace
}  // namespace kq

extern "C" kq_status kq_route_workspace(int64_t rows, int experts, int top, size_t* bytes) {
  using namespace kq;
  const char* fn = "kq_route_workspace";
  if (!bytes) return fail(KQ_EINVAL, "%s: NULL argument", fn);
  KQ_TRY(check_route(fn, (const void*)16, KQ_F32, rows, experts, experts, top, 0));
  int chunks;
  int64_t per;
  deal(rows, experts, &chunks, &per);
  *bytes = round16(sizeof(int32_t) * (size_t)chunks * (experts + 1)) + round16(sizeof(float) * (size_t)chunks * experts) + sizeof(double) * experts;
  return KQ_OK;
}

extern "C" kq_status kq_route(const void* logits, int type, int64_t rows, int experts, int64_t ld, int top, int normalize,
                              float* weight, int32_t* expert, int32_t* slot, int32_t* index, int32_t* offsets,
                              int32_t* counts, float* loss_opt, void* ws, size_t ws_bytes, void* stream) {
  using namespace kq;
  const char* fn = "kq_route";
  KQ_TRY(check_route(fn, logits, type, rows, experts, ld, top, normalize));
  if (rows > 0 && (!weight || !expert || !slot || !index)) return fail(KQ_EINVAL, "%s: NULL output", fn);
  if (!offsets || !counts) return fail(KQ_EINVAL, "%s: NULL offsets or counts", fn);
  if (((uintptr_t)weight | (uintptr_t)expert | (uintptr_t)slot | (uintptr_t)index | (uintptr_t)offsets | (uintptr_t)counts |
       (uintptr_t)loss_opt) & 3)
    return fail(KQ_EINVAL, "%s: an output is not aligned to its type", fn);
  size_t need;
  KQ_TRY(kq_route_workspace(rows, experts, top, &need));
  if (!ws || ws_bytes < need || ((uintptr_t)ws & 15)) return fail(KQ_EWORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
  hipStream_t s = as_stream(stream);
  RouteArgs a{};
  a.logits = logits; a.rows = rows; a.ld = ld; a.experts = experts; a.top = top; a.normalize = normalize;
  a.weight = weight; a.expert = expert; a.slot = slot; a.index = index; a.offsets = offsets; a.counts = counts;
  a.loss = loss_opt;
  deal(rows, experts, &a.chunks, &a.per);
  a.hist = (int32_t*)ws;
  a.prob = (float*)((char*)ws + round16(sizeof(int32_t) * (size_t)a.chunks * (experts + 1)));
  a.mean = (double*)((char*)a.prob + round16(sizeof(float) * (size_t)a.chunks * experts));
  if (rows > 0) KQ_TRY(by_width<RouteRows>(type, experts, RouteLaunch{a, s}));
  route_scan_kernel<<<dim3((unsigned)ceil_div(experts + 1, 16)), dim3(1024), 0, s>>>(a);
  KQ_LAUNCHED("route_scan_kernel");
  const size_t lds = sizeof(int) * ((size_t)(WAVES + 1) * experts + 1);
  if (lds > 64 * 1024)
    KQ_HIP(hipFuncSetAttribute((const void*)route_place_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
  route_place_kernel<<<dim3((unsigned)std::max<int64_t>(1, ceil_div(a.chunks, WAVES))), dim3(64 * WAVES), lds, s>>>(a);
  KQ_LAUNCHED("route_place_kernel");
  return KQ_OK;
}

extern "C" kq_status kq_route_backward(const void* logits, int type, int64_t rows, int experts, int64_t ld, int top,
                                       int normalize, const float* weight, const int32_t* expert, const int32_t* counts,
                                       const float* dweight_opt, const float* dloss_opt, void* dlogits,
                                       int64_t ldd, void* stream) {
  using namespace kq;
  const char* fn = "kq_route_backward";
  KQ_TRY(check_route(fn, logits, type, rows, experts, ld, top, normalize));
  if (ldd < experts) return fail(KQ_ESHAPE, "%s: ldd %lld < %d", fn, (long long)ldd, experts);
  if (rows > 0 && (!weight || !expert || !counts || !dlogits)) return fail(KQ_EINVAL, "%s: NULL argument", fn);
  if (((uintptr_t)weight | (uintptr_t)expert | (uintptr_t)counts | (uintptr_t)dweight_opt | (uintptr_t)dloss_opt) & 3 ||
      (uintptr_t)dlogits & (type == KQ_F32 ? 3 : 1))
    return fail(KQ_EINVAL, "%s: an argument is not aligned to its type", fn);
  if (rows == 0) return KQ_OK;
  BackArgs a{};
  a.logits = logits; a.rows = rows; a.ld = ld; a.ldd = ldd; a.experts = experts; a.top = top; a.normalize = normalize;
  a.weight = weight; a.expert = expert; a.counts = counts; a.dweight = dweight_opt; a.dloss = dloss_opt;
  a.dlogits = dlogits;
  return by_width<RouteBack>(type, experts, BackLaunch{a, as_stream(stream)});
}
