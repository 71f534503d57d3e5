// Routing of rows to a mixture's experts: softmax, the `top` largest logits, slots sorted by expert,
// counts and the balance loss, and the gradient of the logits.
//
// Rows are dealt to workgroups in contiguous chunks, a chunk's rows to its waves likewise.  The first
// kernel takes the softmax and the choices of its rows, counts each wave's choices per expert, and
// leaves every choice's rank among its chunk's at that expert; the second sums the chunks' counts over
// the chunks; the third adds to a rank what lies before its chunk.  Few rows are one chunk, and the
// first kernel does all of it.  Every order is that of the rows, so nothing depends on timing.
#include "device_util.h"
#include "kq_internal.h"
#include "lanes.h"

#include <algorithm>

namespace kq {
namespace {

constexpr int MAX_TOP = 16, MAX_EXPERTS = 4096;
constexpr int MAX_CHUNKS = 1024;
constexpr int PLACERS = 256, BACK_WAVES = 4;   // threads of the third kernel, waves of the gradient's

struct RouteArgs {
  const void* logits;
  int64_t rows, ld;
  int experts, top;
  bool normalize;
  float* weight;
  int32_t* expert;
  int32_t* slot;
  int32_t* index;
  int32_t* offsets;
  int32_t* counts;
  float* loss;
  int chunks;
  int64_t per;            // rows of a wave; a chunk has those of its workgroup's waves
  int32_t* hist;          // [chunks][experts + 1]: choices per expert, rows with a softmax
  float* prob;            // [chunks][experts]: sums of probabilities
  double* mean;           // [experts]: over all chunks
};

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((unsigned)v << 16); }

// exp(x).  The product x log2 e rounds by 2^-24 of itself, a relative error of |x| 2^-24 in the result:
// for the x <= 0 of a softmax largest where the result is least.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(1.44269504f * x); }

// A row's values in registers: LPR lanes hold VPL each, in groups of W = min(VPL, 4) neighbours.
// Value v of lane l is column (v / W) LPR W + l W + v % W, so columns ascend with v in a lane.
template <int LPR, int VPL>
struct Row {
  static constexpr int W = VPL < 4 ? VPL : 4;
  __device__ static constexpr int column(int v) { return v / W * (LPR * W) + v % W; }   // plus W l
};

// W neighbouring values in one access, at any alignment of their type.
template <typename T, int W>
struct Group {
  static constexpr int WORDS = W * (int)sizeof(T) / 4;
  typedef unsigned words __attribute__((ext_vector_type(WORDS > 0 ? WORDS : 1)));
  struct __attribute__((packed, aligned(sizeof(T)))) Memory { words v; };

  __device__ static __forceinline__ float value(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else return bf16_value(v);
  }
  __device__ static __forceinline__ T raw(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else return __builtin_bit_cast(uint16_t, (__bf16)v);
  }
  // Columns c .. c + W - 1 of a row of n, -inf past its end.
  __device__ static __forceinline__ void load(const T* p, int c, int n, float (&r)[W]) {
    if (WORDS > 0 && c + W <= n) {
      const words u = ((const Memory*)(p + c))->v;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(T) == 4) r[i] = __uint_as_float(u[i]);
        else r[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        r[i] = -INFINITY;
        if (c + i < n) r[i] = value(p[c + i]);
      }
    }
  }
  __device__ static __forceinline__ void store(T* p, int c, int n, const float (&r)[W]) {
    if (WORDS > 0 && c + W <= n) {
      words u{};
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(r[i]);
        else u[i / 2] |= (unsigned)raw(r[i]) << (16 * (i & 1));
      }
      ((Memory*)(p + c))->v = u;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (c + i < n) p[c + i] = raw(r[i]);
    }
  }
};

template <typename T, int LPR, int VPL>
__device__ __forceinline__ void load_row(const T* p, int l, int n, float (&r)[VPL]) {
  constexpr int W = Row<LPR, VPL>::W;
#pragma unroll
  for (int g = 0; g < VPL; g += W) {
    float v[W];
    Group<T, W>::load(p, Row<LPR, VPL>::column(g) + W * l, n, v);
#pragma unroll
    for (int i = 0; i < W; ++i) r[g + i] = v[i];
  }
}

// Over the LPR lanes of a row, the result in all of them.
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  return reduce_lanes<LPR>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return reduce_lanes<LPR>(v, [](float a, float b) { return a + b; });
}
template <int LPR>
__device__ __forceinline__ int row_min(int v) {
  return reduce_lanes<LPR>(v, [](int a, int b) { return min(a, b); });
}
template <int LPR>
__device__ __forceinline__ int row_top(int v) {
  return reduce_lanes<LPR>(v, [](int a, int b) { return max(a, b); });
}

// Keys of a row's values: whole numbers in the values' order, whose lowest bits make room for the
// column, counted down, so that they are distinct and the lower of two columns comes first.
// bf16 values keep all their bits; of fp32 values as many go as columns need, and two neighbours
// in the order that agree in the rest have to be compared in full (ambiguous).
constexpr int KEY_FINITE = (int)0x80800000;   // the lowest number's; only -inf (and NaN) lies below
__device__ __forceinline__ int key_of(float v, int column, int low, int mask) {
  const int u = __float_as_int(v);
  return (((u ^ ((u >> 31) & 0x7fffffff)) & ~mask) | low) ^ column;
}

// Sorts N keys, a power of two of them, in descending order: merges of odd and even places, of runs
// of P, at distances Q = P, P / 2, .. 1.
template <int P = 1, int Q = P, int N>
__device__ __forceinline__ void sort_keys(int (&k)[N]) {
  if constexpr (P < N) {
#pragma unroll
    for (int i = Q % P; i + Q < N; ++i)
      if ((i - Q % P) % (2 * Q) < Q && i / (2 * P) == (i + Q) / (2 * P)) {
        const int hi = max(k[i], k[i + Q]), lo = min(k[i], k[i + Q]);
        k[i] = hi;
        k[i + Q] = lo;
      }
    if constexpr (Q > 1)
      sort_keys<P, Q / 2>(k);
    else
      sort_keys<2 * P>(k);
  }
}

// The `count` largest keys of a row, key j to lane j: every lane's are sorted, and the one that holds
// the largest gives it up.  DEPTH: at least count.
template <int LPR, int DEPTH, int J = 0, int N>
__device__ __forceinline__ void take_keys(int (&k)[N], int count, int& mine) {
  if constexpr (J < DEPTH) {
    if (J >= count) return;
    const int best = row_top<LPR>(k[0]);
    if (threadIdx.x % LPR == J) mine = best;
    const bool gives = k[0] == best;
    constexpr int LAST = N - 1, LEFT = DEPTH - 1 - J;   // (as many of a lane's as may still be taken)
#pragma unroll
    for (int i = 0; i < LAST && i < LEFT; ++i) k[i] = gives ? k[i + 1] : k[i];
    if constexpr (LAST < LEFT) k[LAST] = gives ? INT32_MIN : k[LAST];
    take_keys<LPR, DEPTH, J + 1>(k, count, mine);
  }
}

// The rows [r0, r1), by one wave: weights, experts, and each choice's rank among the wave's at its
// expert, in slot; hist (LDS, [experts], zero before) counts the choices; the rows' probabilities are
// added to prob.  Returns its rows with a logit above -inf.
template <typename T, int LPR, int VPL>
__device__ __forceinline__ int route_chunk(const RouteArgs& a, int64_t r0, int64_t r1, int* hist, float (&prob)[VPL]) {
  using R = Row<LPR, VPL>;
  constexpr int ROWS = 64 / LPR;
  const int lane = threadIdx.x & 63, l = lane % LPR;
  int used = 0;
  for (int64_t t = r0; t < r1; t += ROWS) {
    const int64_t row = t + lane / LPR;
    const bool in = row < r1;
    const T* from = (const T*)a.logits + (in ? row : r0) * a.ld;
    float x[VPL];
    load_row<T, LPR, VPL>(from, l, a.experts, x);
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] += 0.f;   // (-0 becomes 0, which it equals)
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
    float total = 0.f, mine = 0.f;
    int chosen = -1;
    // bf16: the keys say it all; fp32: one choice more, to see that the last one is clear of it
    constexpr bool WHOLE = sizeof(T) == 2;
    const int count = a.top + (WHOLE ? 0 : 1);
    bool clear = VPL <= 16 && count <= 16;
    if constexpr (VPL <= 16) {
      if (clear) {
        constexpr int MASK = LPR * VPL - 1;
        const int low = MASK - R::W * l;   // (column(v) has its bits among those of no lane)
        int k[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) k[v] = key_of(x[v], R::column(v), low, MASK);
        int key = INT32_MIN;
        if (count <= 9) {   // (sorted here, since what lies past the ninth is left out of it)
          sort_keys(k);
          take_keys<LPR, 9>(k, count, key);
        } else {
          sort_keys(k);
          take_keys<LPR, 16>(k, count, key);
        }
        const int before = moved<0x111>(key);   // (of the lane before)
        const bool there = key >= KEY_FINITE;
        if (!WHOLE) clear = !__any(l > 0 && l < count && there && ((key ^ before) & ~MASK) == 0);
        if (l < a.top && there && !bad) {
          chosen = MASK - (key & MASK);
          const T v = from[chosen];   // once more, whole
          mine = exp_of((sizeof(T) == 4 ? (float)v : bf16_value((uint16_t)v)) - base);
        }
        total = row_sum<LPR>(mine);
      }
    }
    if (!clear) {
      // one choice after another: the first column of the largest value left
      if constexpr (VPL <= 16) load_row<T, LPR, VPL>(from, l, a.experts, x);   // (not held through the above)
      total = 0.f;
      chosen = -1;
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
    }
    if (in && l < a.top) {
      const float by = a.normalize ? total : sum;
      a.weight[row * a.top + l] = bad ? NAN : chosen >= 0 ? mine / by : 0.f;
      a.expert[row * a.top + l] = chosen;
    }
    // a row's choices are distinct, so row by row no two lanes count at one expert
    int rank = 0;
#pragma unroll
    for (int g = 0; g < ROWS; ++g) {
      if (lane / LPR == g && in && chosen >= 0) {
        rank = hist[chosen];
        hist[chosen] = rank + 1;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // (one lane's view would allow all at once)
      __builtin_amdgcn_wave_barrier();
    }
    if (in && l < a.top) a.slot[row * a.top + l] = rank;
  }
  return used;
}

// Exclusive prefix sums of n counts into first[0 .. n], by one wave.
__device__ __forceinline__ void first_slots(const int* counts, int n, int* first) {
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

// The loss, by all THREADS of a workgroup: sums(e) gives expert e's sum of probabilities.
template <int THREADS, typename F>
__device__ __forceinline__ void write_loss(const RouteArgs& a, const int* first, int used, double* shared, F sums) {
  double s = 0;   // (an expert without choices adds nothing, but a probability that is NaN has to show)
  for (int e = threadIdx.x; e < a.experts; e += THREADS) s += (double)(first[e + 1] - first[e]) * sums(e);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0;
  for (int i = 0; i < THREADS / 64; ++i) s += shared[i];
  *a.loss = (float)(s * a.experts / ((double)max(first[a.experts], 1) * max(used, 1)));
}

// Softmax and choices of a chunk's rows: p_e = exp(l_e - m) / sum exp(l - m), each choice's rank.
// Sixteen lanes a row, so that its reductions are lane rotations, which cost no more than the operation
// (64 lanes past 256 experts).  Bound by the vector instructions: 131072 x 256 fp32, top 8, with the
// loss, 51 us (59 with the logits from memory), VALU busy in four cycles of five, where the logits take 26 at
// 5.2 TB/s (choosing by eight searches for the largest value: 79 us; with the next rows read ahead, which
// spills, 70); one row of eight experts, all of routing in this launch, 4.1 us.
template <typename T, int LPR, int VPL, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void route_rows_kernel(RouteArgs a) {
  using R = Row<LPR, VPL>;
  constexpr int THREADS = 64 * WAVES;
  extern __shared__ __attribute__((aligned(16))) int lds[];   // [WAVES][experts], then of one chunk [experts] and [experts + 1]
  __shared__ int used[WAVES];
  __shared__ double shared[WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = a.experts;
  for (int e = threadIdx.x; e < WAVES * n; e += THREADS) lds[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * WAVES * a.per, r0 = min(c0 + wave * a.per, a.rows), r1 = min(r0 + a.per, a.rows);
  float prob[VPL] = {};
  const int mine = route_chunk<T, LPR, VPL>(a, r0, r1, lds + wave * n, prob);
  if (lane == 0) used[wave] = mine;
  __syncthreads();
  // counts of the waves before, and of the chunk
  int* total = lds + WAVES * n;
  int* first = total + n;
  const bool one = gridDim.x == 1;
  int32_t* to = a.hist + (int64_t)blockIdx.x * (n + 1);
  for (int e = threadIdx.x; e < n; e += THREADS) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int v = lds[w * n + e];
      lds[w * n + e] = sum;
      sum += v;
    }
    if (one)
      total[e] = a.counts[e] = sum;
    else
      to[e] = sum;
  }
  int all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) all += used[w];
  if (threadIdx.x == 0) *(one ? a.counts + n + 1 : to + n) = all;
  __syncthreads();
  if (one) {
    if (wave == 0) first_slots(total, n, first);
    __syncthreads();
    for (int e = threadIdx.x; e <= n; e += THREADS) a.offsets[e] = first[e];
    if (threadIdx.x == 0) a.counts[n] = first[n];
    for (int64_t i = first[n] + threadIdx.x; i < a.rows * a.top; i += THREADS) a.index[i] = -1;
  }
  // each wave its own rows' choices (which it has written)
  for (int64_t i = r0 * a.top + lane; i < r1 * a.top; i += 64) {
    const int e = a.expert[i];
    if (e < 0) {
      a.slot[i] = -1;
      continue;
    }
    const int rank = a.slot[i] + lds[wave * n + e];
    if (one) {
      a.slot[i] = first[e] + rank;
      a.index[first[e] + rank] = (int32_t)((uint32_t)i / (uint32_t)a.top);
    } else {
      a.slot[i] = rank;
    }
  }
  if (!a.loss) return;
  // the waves' probabilities, summed in their order
  __syncthreads();
  float* sums = (float*)lds + wave * n;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float s = prob[v];
    if constexpr (LPR == 16) {
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
    }
    const int c = R::column(v) + R::W * (lane % LPR);
    if (lane < LPR && c < n) sums[c] = s;
  }
  __syncthreads();
  auto sum_of = [&](int e) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += ((const float*)lds)[w * n + e];
    return s;
  };
  if (one)
    write_loss<THREADS>(a, first, all, shared, sum_of);
  else
    for (int e = threadIdx.x; e < n; e += THREADS) a.prob[(int64_t)blockIdx.x * n + e] = sum_of(e);
}

// Eight experts (and, past the last, the count of rows) per workgroup, 128 threads each: the chunks'
// counts become those of the chunks before, the totals go to counts, the probabilities' sums (in 64
// bits from here on) to mean.  Every thread's reads are out before it adds, so that one trip to memory
// and one back are all there is: 1024 chunks of 256 experts 8.6 us, 17 workgroups that read one chunk
// after another 28.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteArgs a) {
  constexpr int SEGS = 128, PER = MAX_CHUNKS / SEGS;
  __shared__ int seg[8][SEGS + 1];
  __shared__ double seg_p[8][SEGS + 1];
  const int k = threadIdx.x & 7, s = threadIdx.x >> 3, e = blockIdx.x * 8 + k;
  const int64_t pitch = a.experts + 1;
  const int per = (a.chunks + SEGS - 1) / SEGS, c0 = s * per;
  const bool live = e <= a.experts, summed = e < a.experts && a.loss;
  int v[PER], n = 0;
  float f[PER];
  double p = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = live && i < per && c0 + i < a.chunks ? a.hist[(c0 + i) * pitch + e] : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) f[i] = summed && i < per && c0 + i < a.chunks ? a.prob[(int64_t)(c0 + i) * a.experts + e] : 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    n += v[i];
    p += f[i];
  }
  seg[k][s] = n;
  seg_p[k][s] = p;
  __syncthreads();
  // one wave per expert: two segments a lane
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (wave < 8) {
    const int x = seg[wave][2 * lane], y = seg[wave][2 * lane + 1];
    int sum = x + y;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o);
      if (lane >= o) sum += u;
    }
    double q = seg_p[wave][2 * lane] + seg_p[wave][2 * lane + 1];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) q += __shfl_xor(q, o);
    seg[wave][2 * lane] = sum - x - y;
    seg[wave][2 * lane + 1] = sum - y;
    const int mine = blockIdx.x * 8 + wave;
    if (lane == 63 && mine <= a.experts) {
      a.counts[mine == a.experts ? mine + 1 : mine] = sum;
      if (mine < a.experts && a.loss) a.mean[mine] = q;
    }
  }
  __syncthreads();
  int before = seg[k][s];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (e < a.experts && i < per && c0 + i < a.chunks) {
      a.hist[(c0 + i) * pitch + e] = before;
      before += v[i];
    }
}

// Slots: an expert's first one, the choices of the chunks before, the rank in the chunk.  Latency, and
// scattered writes of the index: 131072 rows of 8 choices 9.6 us, 4099 of 6 5.1 with the counts' sums.
// SCANNED: the second kernel has been; else every workgroup adds up the chunks' counts itself.
template <bool SCANNED>
__global__ __launch_bounds__(PLACERS) void route_place_kernel(RouteArgs a, int64_t chunk_rows) {
  extern __shared__ int lds[];   // first slots [experts + 1], the chunk's next ones [experts]
  __shared__ double shared[PLACERS / 64];
  __shared__ int sums[PLACERS / 64];
  __shared__ int all[SCANNED ? 1 : PLACERS], earlier_of[SCANNED ? 1 : PLACERS];
  __shared__ double part[SCANNED ? 1 : PLACERS];
  const int n = a.experts, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* next = lds + n + 1;
  const int32_t* before = a.hist + (int64_t)blockIdx.x * (n + 1);
  const int64_t choices = a.rows * a.top, i0 = blockIdx.x * chunk_rows * a.top, i1 = min(i0 + chunk_rows * a.top, choices);
  // the first choices are on their way while the first slots are summed
  constexpr int EARLY = 4;
  int early_e[EARLY], early_r[EARLY];
#pragma unroll
  for (int k = 0; k < EARLY; ++k) {
    const int64_t i = i0 + k * PLACERS + threadIdx.x;
    early_e[k] = i < i1 ? a.expert[i] : -1;
    early_r[k] = i < i1 ? a.slot[i] : 0;
  }
  int used = 0;
  if constexpr (!SCANNED) {
    // thread (g, e) takes every groups-th chunk's count at expert e
    const int groups = PLACERS / n, g = threadIdx.x / n, e = threadIdx.x % n;
    all[threadIdx.x] = earlier_of[threadIdx.x] = 0;
    __syncthreads();
    if (g < groups) {
      int total = 0, mine = 0;
#pragma unroll 8
      for (int c = g; c < a.chunks; c += groups) {
        const int v = a.hist[(int64_t)c * (n + 1) + e];
        total += v;
        mine += c < (int)blockIdx.x ? v : 0;
      }
      atomicAdd(all + e, total);
      atomicAdd(earlier_of + e, mine);
    }
    if (blockIdx.x == 0) {   // what the second kernel leaves in counts and mean
      if (a.loss && g < groups) {
        double p = 0;
#pragma unroll 8
        for (int c = g; c < a.chunks; c += groups) p += a.prob[(int64_t)c * n + e];
        part[threadIdx.x] = p;
      }
      for (int c = threadIdx.x; c < a.chunks; c += PLACERS) used += a.hist[(int64_t)c * (n + 1) + n];
      used = reduce_lanes<64>(used, [](int x, int y) { return x + y; });
      if (lane == 0) sums[wave] = used;
      __syncthreads();
      used = 0;
#pragma unroll
      for (int w = 0; w < PLACERS / 64; ++w) used += sums[w];
      if (a.loss && threadIdx.x < n) {
        double p = 0;
        for (int i = 0; i < groups; ++i) p += part[i * n + threadIdx.x];
        a.mean[threadIdx.x] = p;
      }
      if (threadIdx.x < n) a.counts[threadIdx.x] = all[threadIdx.x];
      if (threadIdx.x == 0) a.counts[n + 1] = used;
    }
    __syncthreads();
  }
  int base = 0;
  for (int e0 = 0; e0 < n; e0 += PLACERS) {
    const int e = e0 + threadIdx.x;
    int c = 0, earlier = 0;
    if (e < n) {
      c = SCANNED ? a.counts[e] : all[SCANNED ? 0 : e];
      earlier = SCANNED ? before[e] : earlier_of[SCANNED ? 0 : e];
    }
    int sum = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    int first = base + sum - c;
#pragma unroll
    for (int w = 0; w < PLACERS / 64; ++w) {
      if (w < wave) first += sums[w];
      base += sums[w];
    }
    if (e < n) {
      lds[e] = first;
      next[e] = first + earlier;
    }
    __syncthreads();
  }
  const int made = base;
  if (threadIdx.x == 0) lds[n] = made;
  auto put = [&](int64_t i, int e, int rank) {
    if (e < 0) return;   // (its slot is -1 already)
    const int slot = next[e] + rank;
    a.slot[i] = slot;
    a.index[slot] = (int32_t)((uint32_t)i / (uint32_t)a.top);
  };
#pragma unroll
  for (int k = 0; k < EARLY; ++k) put(i0 + k * PLACERS + threadIdx.x, early_e[k], early_r[k]);
  for (int64_t i = i0 + EARLY * PLACERS + threadIdx.x; i < i1; i += PLACERS) put(i, a.expert[i], a.slot[i]);
  for (int64_t i = max((int64_t)made, i0) + threadIdx.x; i < i1; i += PLACERS) a.index[i] = -1;
  if (blockIdx.x != 0) return;
  __syncthreads();
  for (int e = threadIdx.x; e <= n; e += PLACERS) a.offsets[e] = lds[e];
  if (threadIdx.x == 0) a.counts[n] = made;
  if (a.loss) write_loss<PLACERS>(a, lds, SCANNED ? a.counts[n + 1] : used, shared, [&](int e) { return a.mean[e]; });
}

// What the wave's lanes have written to LDS before is what they read after.
__device__ __forceinline__ void wave_step() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct BackArgs {
  const void* logits;
  int64_t rows, ld, ldd;
  int experts, top;
  bool normalize;
  const float* weight;
  const int32_t* expert;
  const int32_t* counts;
  const float* dweight;
  const float* dloss;
  void* dlogits;
  int64_t per;
};

// The logits' gradient, dl_e = p_e (b_e - back) + [e chosen] extra, by the lanes that hold the row.
// Bound by HBM: 131072 x 256 fp32, top 8, 55 us, 5.1 TB/s (each lane comparing its columns with every
// choice: 61 us, and 48 for the bf16 that takes 32 so).
template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(64 * BACK_WAVES) void route_backward_kernel(BackArgs a) {
  using R = Row<LPR, VPL>;
  constexpr int ROWS = 64 / LPR;
  struct alignas(4 * R::W) Part { float v[R::W]; };
  __shared__ __attribute__((aligned(16))) float parts[BACK_WAVES][ROWS][LPR * VPL];
  const int lane = threadIdx.x & 63, l = lane % LPR;
  float* mine = parts[threadIdx.x >> 6][lane / LPR];
#pragma unroll
  for (int v = 0; v < VPL; ++v) mine[v * LPR + l] = 0.f;
  wave_step();
  const int64_t chunk = (int64_t)blockIdx.x * BACK_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    load_row<T, LPR, VPL>((const T*)a.logits + from * a.ld, l, a.experts, x);
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
    const bool none = sum == 0.f;   // (no logit above -inf)
    const float inv = 1.f / sum;
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
    for (int v = 0; v < VPL; ++v) x[v] = none ? 0.f : x[v] * (b[v] - back);   // (zero beside a dloss of inf or NaN too)
    if (a.dweight) {
      // the chosen columns' part goes to the lanes that hold them through LDS, which is zero else
      const bool adds = l < a.top && chosen >= 0 && chosen < a.experts;
      if (adds) mine[chosen] = extra;
      wave_step();
#pragma unroll
      for (int v = 0; v < VPL; v += R::W) {
        const Part p = *(const Part*)(mine + R::column(v) + R::W * l);
#pragma unroll
        for (int i = 0; i < R::W; ++i) x[v + i] += p.v[i];
      }
      wave_step();
      if (adds) mine[chosen] = 0.f;
      wave_step();
    }
    if (!in) continue;
    T* to = (T*)a.dlogits + row * a.ldd;
#pragma unroll
    for (int v = 0; v < VPL; v += R::W) {
      float out[R::W];
#pragma unroll
      for (int i = 0; i < R::W; ++i) out[i] = x[v + i];
      Group<T, R::W>::store(to, R::column(v) + R::W * l, a.experts, out);
    }
  }
}

// Waves of a workgroup of the first kernel: eight, four where their counts would take more LDS.
int waves_of(int experts) { return experts <= 2048 ? 8 : 4; }

// The rows of a wave and the number of chunks: few rows are one (64 of 256 experts: 11.7 us, in chunks of
// 32 rows 13.7, 128 of them 17.4 and 14.0; 128 of 8 experts 8.1 and 10.1), then one for each compute unit
// until a wave has sixteen rows (32768 of 64 experts: 19 us, with four rows a wave 22; 4099 of them 12.7,
// with sixteen 16.5).
void deal(int64_t rows, int experts, int* chunks, int64_t* per) {
  const int64_t waves = waves_of(experts);
  auto share = [&](int64_t n) { return ceil_div(ceil_div(rows, n * waves), 4) * 4; };
  *per = rows <= (experts <= 64 ? 128 : 64) ? share(1) : std::max(std::min<int64_t>(share(256), 16), share(MAX_CHUNKS));
  *per = std::max<int64_t>(*per, 4);
  *chunks = (int)std::max<int64_t>(ceil_div(rows, *per * waves), 1);
}

// The most chunks that deal() makes of up to so many rows (its own number does not always grow with them).
int64_t most_chunks(int64_t rows, int experts) {
  const int64_t waves = waves_of(experts);
  return std::min(std::min<int64_t>(MAX_CHUNKS, ceil_div(rows, 4 * waves)), std::max<int64_t>(256, ceil_div(rows, 16 * waves)));
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
    constexpr int WAVES = LPR * VPL <= 2048 ? 8 : 4;
    RouteArgs a = r.a;
    const size_t lds = sizeof(int) * ((size_t)(WAVES + 2) * a.experts + 1);
    const auto kernel = route_rows_kernel<T, LPR, VPL, WAVES>;
    if (lds > 64 * 1024 - 256)   // (beside it `used` and `shared`, up to 96 bytes)
      KQ_HIP(hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds));
    kernel<<<dim3((unsigned)a.chunks), dim3(64 * WAVES), lds, r.s>>>(a);
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
    const int64_t units = ceil_div(a.rows, 64 / LPR), waves = std::min<int64_t>(units, (int64_t)device_cu_count() * 32);
    a.per = ceil_div(units, waves) * (64 / LPR);
    const unsigned grid = (unsigned)ceil_div(ceil_div(a.rows, a.per), BACK_WAVES);
    route_backward_kernel<T, LPR, VPL><<<dim3(grid), dim3(64 * BACK_WAVES), 0, r.s>>>(a);
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
  const size_t most = (size_t)most_chunks(rows, experts);
  *bytes = chunks == 1 ? 0 : round16(sizeof(int32_t) * most * (experts + 1)) + round16(sizeof(float) * most * experts) + sizeof(double) * experts;
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
  if (need > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 15))) return fail(KQ_EWORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
  hipStream_t s = as_stream(stream);
  RouteArgs a{};
  a.logits = logits; a.rows = rows; a.ld = ld; a.experts = experts; a.top = top; a.normalize = normalize;
  a.weight = weight; a.expert = expert; a.slot = slot; a.index = index; a.offsets = offsets; a.counts = counts;
  a.loss = loss_opt;
  deal(rows, experts, &a.chunks, &a.per);
  a.hist = (int32_t*)ws;   // (one chunk has no use for it)
  a.prob = (float*)((char*)ws + round16(sizeof(int32_t) * (size_t)a.chunks * (experts + 1)));
  a.mean = (double*)((char*)a.prob + round16(sizeof(float) * (size_t)a.chunks * experts));
  KQ_TRY(by_width<RouteRows>(type, experts, RouteLaunch{a, s}));
  if (a.chunks == 1) return KQ_OK;
  // Few counts are added up by every workgroup that needs them, which spares a launch, of about 3.5 us for
  // the caller (2048 rows of 64 experts, 4096 counts: 11.1 us on the GPU, through the second kernel 11.9;
  // 8192 of 32, 8192 counts: 12.4 and 12.3; 8192 of 64, 16384 counts: 15.7 and 13.4).
  const bool scanned = experts > PLACERS || (int64_t)a.chunks * experts > 10000;
  if (scanned) {
    route_scan_kernel<<<dim3((unsigned)ceil_div(experts + 1, 8)), dim3(1024), 0, s>>>(a);
    KQ_LAUNCHED("route_scan_kernel");
  }
  const auto place = scanned ? route_place_kernel<true> : route_place_kernel<false>;
  place<<<dim3((unsigned)a.chunks), dim3(PLACERS), sizeof(int) * (2 * (size_t)experts + 1), s>>>(a, a.per * waves_of(experts));
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
  if (dlogits == logits && ldd != ld) return fail(KQ_EINVAL, "%s: in place, ldd is ld", fn);
  if (rows == 0) return KQ_OK;
  BackArgs a{};
  a.logits = logits; a.rows = rows; a.ld = ld; a.ldd = ldd; a.experts = experts; a.top = top; a.normalize = normalize;
  a.weight = weight; a.expert = expert; a.counts = counts; a.dweight = dweight_opt; a.dloss = dloss_opt;
  a.dlogits = dlogits;
  return by_width<RouteBack>(type, experts, BackLaunch{a, as_stream(stream)});
}
