// Products with layers held in MXFP4: y = Q(x~) W^T for one layer, or for one of several
// layers per row (a mixture's experts), sums in fp32 on the scaled matrix instructions.
#include "mxfp4_tiles.h"

#include <algorithm>

namespace kq {
namespace {

// Where a tile's rows of x come from: consecutive rows, rows behind an index, or rows behind an
// index of an x too large for 32-bit offsets.
enum { X_ROWS, X_INDEX, X_FAR };

// Experts whose tiles a kernel finds through its table; more are searched in memory.
constexpr int TABLE = 1024;
struct ExpertTable {
  int before[TABLE];      // row tiles of the experts before this one
  int first[TABLE + 1];   // its first slot; of the one past the last: the end
};

// Row tiles of all experts; with at most TABLE experts, the table too (all threads of the
// workgroup, which a barrier has to follow).
template <int BM>
__device__ __forceinline__ int count_tiles(const ProductArgs& a, ExpertTable& tab) {
  const int lane = threadIdx.x & 63;
  int tm = 0;
  for (int e0 = 0, top = 0; e0 < a.experts; e0 += 64) {
    int first, last;
    expert_ranges(a, e0, top, first, last);
    const int c = (last - first + BM - 1) / BM;
    int sum = c;   // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o);
      if (lane >= o) sum += v;
    }
    if (a.experts <= TABLE && threadIdx.x < 64 && e0 + lane < a.experts) {
      tab.before[e0 + lane] = tm + sum - c;
      tab.first[e0 + lane] = first;
      if (e0 + lane == a.experts - 1) tab.first[a.experts] = last;
    }
    tm += __builtin_amdgcn_readlane(sum, 63);
  }
  if (a.experts <= TABLE && threadIdx.x < 64)
    for (int e = a.experts + lane; e < TABLE; e += 64) tab.before[e] = 0x7fffffff;
  return __builtin_amdgcn_readfirstlane(tm);
}

// The expert of row tile mt (< the count) and the tile's rows.
template <int BM>
__device__ __forceinline__ void find_rows(const ProductArgs& a, const ExpertTable& tab, int mt, Tile& t) {
  const int lane = threadIdx.x & 63;
  if (a.experts <= TABLE) {
    // the last expert with before <= mt: it has tiles, or the next one would have the same before
    const int b = 16 * (__popcll(__ballot(tab.before[16 * lane] <= mt)) - 1);
    const int e = b + __popcll(__ballot(lane < 16 && tab.before[b + (lane & 15)] <= mt)) - 1;
    t.e = __builtin_amdgcn_readfirstlane(e);
    t.m0 = __builtin_amdgcn_readfirstlane(tab.first[t.e] + (mt - tab.before[t.e]) * BM);
    t.last = __builtin_amdgcn_readfirstlane(tab.first[t.e + 1]);
    return;
  }
  search_rows<BM>(a, mt, t);
}

// Tile `id` of tm x tn, counted in bands of G row tiles so that neighbours share panels.
template <int BM, int BN, int G, int ROWS>
__device__ __forceinline__ Tile tile_at(const ProductArgs& a, const ExpertTable& tab, int64_t id, int tm, int tn) {
  const int64_t band = (int64_t)G * tn;
  const int g = (int)(id / band), rem = (int)(id - g * band);
  const int gs = min(G, tm - g * G), mt = g * G + rem % gs;
  Tile t;
  t.n0 = rem / gs * BN;
  if (ROWS == X_ROWS) {
    t.e = 0;
    t.m0 = mt * BM;
    t.last = (int)a.slots;
  } else {
    find_rows<BM>(a, tab, mt, t);
  }
  // (the same for every lane; said here, or each copy would loop over its lanes' descriptors)
  return Tile{__builtin_amdgcn_readfirstlane(t.e), __builtin_amdgcn_readfirstlane(t.m0),
              __builtin_amdgcn_readfirstlane(t.last), __builtin_amdgcn_readfirstlane(t.n0)};
}

// A word of LDS that a copy has put there, once the caller knows it has landed: behind a plain
// read the compiler would wait for every copy and store outstanding.
__device__ __forceinline__ int read_lds(const int* p) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(v) : "v"((unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)p) : "memory");
  return v;
}

// One wave's copy of 64 pieces of SIZE bytes into LDS, piece l to `to` + SIZE l; a lane whose
// offset lies outside the descriptor copies zeros.
template <int SIZE>
__device__ __forceinline__ void copy_lds(__amdgpu_buffer_rsrc_t r, unsigned off, uint8_t* to) {
  typedef __attribute__((address_space(3))) void lds_void;
  if constexpr (SIZE == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, (int)off, 0, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, (int)off, 0, 0, 0);
}
template <int SIZE>
__device__ __forceinline__ void copy_lds(const uint8_t* from, uint8_t* to) {
  typedef __attribute__((address_space(3))) void lds_void;
  if constexpr (SIZE == 16)
    __builtin_amdgcn_global_load_lds((const void*)from, (lds_void*)to, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds((const void*)from, (lds_void*)to, 4, 0, 0);
}

// Stores W values side by side at byte offset `off` (a masked offset stores nothing).
template <int W>
__device__ __forceinline__ void store_f32(__amdgpu_buffer_rsrc_t r, int off, const float (&v)[W]) {
  if constexpr (W == 4)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                 __float_as_uint(v[3])}, r, off, 0, 0);
  else if constexpr (W == 2)
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])}, r, off, 0, 0);
  else
    bstore(v[0], r, off);
}
template <int W>
__device__ __forceinline__ void store_bf16(__amdgpu_buffer_rsrc_t r, int off, const float (&v)[W]) {
  if constexpr (W == 4)
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, r, off, 0, 0);
  else if constexpr (W == 2)
    __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(v[0], v[1]), r, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b16(to_bf16(v[0]), r, off, 0, 0);
}

// Tiles of BM x BN outputs, 256 of K per stage, waves in 2 x WC, each with MT x NT accumulators
// of 32 x 32.  A stage is 128 bytes of every row, a whole line: with 64, the
// copies alone of an 8192 x 8192 x 8192 product took 170 us, with 128 107 us.  A workgroup takes
// tile after tile; the copies of the next tile's first stages follow those of the last stages of
// the present one, so the ring never runs dry and the stores of one tile go out while the next is
// multiplied.
// 16384 x 8192 x 28672: 1.78 ms, 4.3 PF, the matrix instructions busy 68 % of the time at 1.55 GHz
// (alone, from registers, they are held to 1.56 GHz by power: 6.4 PF); eight waves of 128 x 64,
// since four of 128 x 128, which read a third less from LDS, are 2 % slower.  2048 x 11008 x 4096 with
// 128 x 128 tiles: 55 us, 3.3 PF; with 256 x 256, on half as many workgroups, 71.
// RING: stages in LDS; four where a tile is small (256 x 10496 x 2914: 14 us, with two and more
// workgroups side by side 21).
template <int MT, int NT, int WC, int RING, int ROWS>
__global__ __launch_bounds__(128 * WC, WC == 4 ? 2 : 1) void mx_tile_kernel(ProductArgs a) {
  constexpr int BM = 64 * MT, BN = 32 * NT * WC, PANEL_A = BM * 128, PANELS = (BM + BN) * 128;
  constexpr int CA = 4 * MT / WC, CB = 2 * NT;        // copies of x and of W per wave and stage
  constexpr int SI = (BM + BN) / 64, SC = (SI + 2 * WC - 1) / (2 * WC);   // scale copies of 128 of K: all, per wave
  constexpr int COPIES = CA + CB + 2 * SC, SCALES = (BM + BN) * 4;
  constexpr int STAGE = PANELS + 2 * SCALES;
  constexpr bool DEEP = MT * NT < 8;   // registers for the operands of all four quarters of a stage
  __shared__ __attribute__((aligned(1024))) uint8_t b0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t b1[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t b2[RING == 4 ? STAGE : 1024];
  __shared__ __attribute__((aligned(1024))) uint8_t b3[RING == 4 ? STAGE : 1024];
  __shared__ ExpertTable tab[1];
  __shared__ __attribute__((aligned(256))) int next_index[ROWS == X_ROWS ? 64 : BM];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC, l32 = lane & 31, q = lane >> 5;

  // Workgroup u runs on XCD u mod 8 (a heuristic: any order is right).  Each XCD takes a
  // contiguous run of tiles, so that those resident on it at a time share panels in its L2.
  int tm = (int)((a.slots + BM - 1) / BM);
  if (ROWS != X_ROWS) {
    tm = count_tiles<BM>(a, *tab);
    __syncthreads();
  }
  const int tn = (int)((a.N + BN - 1) / BN), turns = gridDim.x >> 3;
  const int64_t total = (int64_t)tm * tn, per = (total + 7) / 8, run = (blockIdx.x & 7) * per;
  const int64_t end = min(run + per, total);
  int64_t id = run + (blockIdx.x >> 3);
  if (id >= end) return;
  auto at_id = [&](int64_t k) { return tile_at<BM, BN, 4, ROWS>(a, *tab, k, tm, tn); };

  // Copies: descriptors whose base advances a stage at a time, and each lane's offset from it.
  // Lanes of rows outside x, and past the last column all copies of x, lie outside their
  // descriptor and put zeros into LDS.
  constexpr unsigned ALL = 0xfffffff0u;
  const uint8_t *xc, *xs, *wc_e, *ws_e;
  unsigned oa[CA], ob[CB], os[SC];   // (X_FAR: os holds rows)
  const uint8_t* pa[CA];   // X_FAR: x beyond the reach of a 32-bit offset
  int stepa[CA];
  int issued;
  // Points the copies at tile t; `row` gives the row of x behind a row of the tile.
  auto aim = [&](const Tile& t, auto row_of_x) {
    auto x_row = [&](int r) -> int64_t {   // -1: zeros
      if (ROWS == X_ROWS) return min(r, t.last - 1 - t.m0);
      const int x = row_of_x(min(r, t.last - 1 - t.m0));
      return x >= 0 && x < a.rows ? x : -1;
    };
    auto w_row = [&](int r) -> unsigned { return (unsigned)min((int64_t)r, a.N - 1 - t.n0); };
    issued = 0;
    int ln = lane;
    asm volatile("" : "+v"(ln));   // the positions computed here, not kept in registers for every tile
    xc = a.xc + (ROWS == X_ROWS ? t.m0 * a.pitch : 0);
    xs = a.xs + (ROWS == X_ROWS ? (int64_t)t.m0 * 4 : 0);
    wc_e = a.wc + ((int64_t)t.e * a.N + t.n0) * a.pitch;
    ws_e = a.ws + (int64_t)t.e * a.N * (4 * a.steps) + (int64_t)t.n0 * 4;
#pragma unroll
    for (int r = 0; r < CA; ++r) {
      const int pos = (wave * CA + r) * 8 + (ln >> 3), p = pos % (32 * MT);
      const int64_t row = x_row(pos / (32 * MT) * (32 * MT) + (p & 31) * MT + (p >> 5));
      const int64_t at = row * a.pitch + 16 * ((ln & 7) ^ ((pos >> 1) & 7));
      oa[r] = row >= 0 ? (unsigned)at : ALL;
      pa[r] = row >= 0 ? a.xc + at : (const uint8_t*)g_zeros;
      stepa[r] = row >= 0 ? 128 : 0;
    }
#pragma unroll
    for (int r = 0; r < CB; ++r) {
      const int pos = (wave * CB + r) * 8 + (ln >> 3), p = pos % (32 * NT);
      ob[r] = w_row(pos / (32 * NT) * (32 * NT) + (p & 31) * NT + (p >> 5)) * (unsigned)a.pitch +
              16 * ((ln & 7) ^ ((pos >> 1) & 7));
    }
#pragma unroll
    for (int k = 0; k < SC; ++k) {
      const int si = min(wave * SC + k, SI - 1);
      const int64_t row = si < MT ? x_row(64 * si + ln) : w_row(64 * (si - MT) + ln);
      os[k] = row >= 0 ? (unsigned)row * (ROWS == X_FAR ? 1 : 4) : ALL;
    }
  };
  const int stages = (a.steps + 1) / 2;
  auto issue = [&](uint8_t* buf) {
    // The last stage of an odd number of steps has no second half: its lanes leave their
    // descriptors.  (In the swizzled order a lane's half of the row is that of its source.)
    const bool live = issued < stages, half = (a.steps & 1) && issued >= stages - 1;
    const __amdgpu_buffer_rsrc_t ra = rsrc(xc, live ? (int)ALL : 0), rb = rsrc(wc_e, (int)ALL);
#pragma unroll
    for (int r = 0; r < CA; ++r) {
      uint8_t* to = buf + (wave * CA + r) * 1024;
      const bool cut = half && (((lane & 7) ^ (((wave * CA + r) * 8 + (lane >> 3)) >> 1)) & 4);
      if (ROWS == X_FAR) {
        copy_lds<16>(live && !cut ? pa[r] : (const uint8_t*)g_zeros, to);
        pa[r] += stepa[r];
      } else {
        copy_lds<16>(ra, cut ? ALL : oa[r], to);
      }
    }
#pragma unroll
    for (int r = 0; r < CB; ++r) {
      const bool cut = half && (((lane & 7) ^ (((wave * CB + r) * 8 + (lane >> 3)) >> 1)) & 4);
      copy_lds<16>(rb, cut ? ALL : ob[r], buf + PANEL_A + (wave * CB + r) * 1024);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < SC; ++k) {
        const int si = min(wave * SC + k, SI - 1);
        const uint8_t* from = si < MT ? xs + 4 * a.rows * h : ws_e + 4 * a.N * h;
        uint8_t* to = buf + PANELS + h * SCALES + si * 256;
        if (ROWS == X_FAR)   // (four bytes of 2^30 rows: the last offsets would be the masked ones)
          copy_lds<4>(os[k] != ALL && !(h && half) ? from + 4 * (uint64_t)os[k] : (const uint8_t*)g_zeros, to);
        else
          copy_lds<4>(rsrc(from, h && half ? 0 : (int)ALL), os[k], to);
      }
    // past the end the last stage's weights and scales are copied again, with zeros for x
    const int64_t on = ++issued < stages;
    xc += 128 * on;
    wc_e += 128 * on;
    xs += 8 * a.rows * on;
    ws_e += 8 * a.N * on;
  };

  f32x16 acc[MT][NT];

  // operands of 64 of K, quarter h of a stage: the lane's row, its chunk 2 h + q of 16 bytes, which
  // lies in the place with the row's bits 1 .. 3 flipped (so that 16 rows cover all banks)
  const int off0 = l32 * 128 + (q ^ ((l32 >> 1) & 7)) * 16;
  const int sca = PANELS + (wr * 32 * MT + l32 * MT) * 4, scb = PANELS + BM * 4 + (wc * 32 * NT + l32 * NT) * 4;
  auto read = [&](const uint8_t* buf, int h, i32x4 (&xa)[MT], i32x4 (&xb)[NT]) {
    const int off = off0 ^ (32 * h);
    const uint8_t* pA = buf + wr * MT * 4096 + off;
    const uint8_t* pB = buf + PANEL_A + wc * NT * 4096 + off;
    xa[0] = *(const i32x4*)pA;
#pragma unroll
    for (int n = 0; n < NT; ++n) xb[n] = *(const i32x4*)(pB + n * 4096);
#pragma unroll
    for (int m = 1; m < MT; ++m) xa[m] = *(const i32x4*)(pA + m * 4096);
  };
  auto read_scales = [&](const uint8_t* buf, int h, int (&sa)[MT], int (&sb)[NT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] = *(const int*)(buf + h * SCALES + sca + 4 * m);
#pragma unroll
    for (int n = 0; n < NT; ++n) sb[n] = *(const int*)(buf + h * SCALES + scb + 4 * n);
  };
  // The lane's bytes of them: where they are used, not where they are read, since that would wait.
  auto own_bytes = [&](int (&sa)[MT], int (&sb)[NT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] >>= 8 * q;
#pragma unroll
    for (int n = 0; n < NT; ++n) sb[n] >>= 8 * q;
  };
  auto mma0 = [&](const i32x4 (&xa)[MT], const i32x4 (&xb)[NT], const int (&sa)[MT], const int (&sb)[NT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(xa[m]), widen(xb[n]), acc[m][n], 4, 4, 0,
                                                                   sa[m], 0, sb[n]);
  };
  auto mma1 = [&](const i32x4 (&xa)[MT], const i32x4 (&xb)[NT], const int (&sa)[MT], const int (&sb)[NT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(xa[m]), widen(xb[n]), acc[m][n], 4, 4, 2,
                                                                   sa[m], 2, sb[n]);
  };

  Tile t = at_id(id);
  aim(t, [&](int r) { return a.index ? a.index[t.m0 + r] : t.m0 + r; });
  i32x4 xa[MT], xb[NT], ya[MT], yb[NT];
  int sa[MT], sb[NT], ta[MT], tb[NT];
  issue(b0);
  issue(b1);
  if constexpr (RING == 4) {
    issue(b2);
    issue(b3);
  }
  __builtin_amdgcn_s_waitcnt(wait_vm((RING - 1) * COPIES));
  lds_barrier();
  read(b0, 0, xa, xb);
  read_scales(b0, 0, sa, sb);
  i32x4 za[MT], zb[NT], ua[MT], ub[NT];
  if constexpr (DEEP) read(b0, 1, ya, yb);

// Stage: read the operands of each quarter while multiplying the one before.  Ahead of the last
// quarter, wait for this wave's copies of the next stage and for every wave's reads of this one;
// then refill its buffer and read the next stage's first quarter.  DEEP: by halves, so that a read
// has two quarters to arrive (2048 x 11008 x 4096, 128 x 128 tiles: 57 -> 55 us; the 256 x 256 tiles'
// accumulators leave no room).
#define KQ_MX_SPREAD(COUNT, GROUP)                          \
  _Pragma("unroll") for (int i_ = 0; i_ < (COUNT); ++i_) {  \
    __builtin_amdgcn_sched_group_barrier(0x008, 1, GROUP);  \
    __builtin_amdgcn_sched_group_barrier(0x100, 2, GROUP);  \
  }                                                         \
  __builtin_amdgcn_sched_barrier(0);
#define KQ_MX_STAGE(CUR, NXT, WAIT)                         \
  {                                                         \
    own_bytes(sa, sb);                                      \
    read(CUR, 1, ya, yb);                                   \
    mma0(xa, xb, sa, sb);                                   \
    KQ_MX_SPREAD(MT + NT, 0)                                \
    read_scales(CUR, 1, ta, tb);                            \
    read(CUR, 2, xa, xb);                                   \
    mma1(ya, yb, sa, sb);                                   \
    KQ_MX_SPREAD(MT + NT + 2, 0)                            \
    own_bytes(ta, tb);                                      \
    read(CUR, 3, ya, yb);                                   \
    mma0(xa, xb, ta, tb);                                   \
    KQ_MX_SPREAD(MT + NT, 0)                                \
    WAIT;                                                   \
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);                 \
    lds_barrier();                                          \
    issue(CUR);                                             \
    read_scales(NXT, 0, sa, sb);                            \
    read(NXT, 0, xa, xb);                                   \
    mma1(ya, yb, ta, tb);                                   \
    _Pragma("unroll") for (int i_ = 0; i_ < MT * NT; ++i_) { \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);    \
      __builtin_amdgcn_sched_group_barrier(0x020, (COPIES + MT * NT - 1) / (MT * NT), 1); \
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);    \
    }                                                       \
    __builtin_amdgcn_sched_barrier(0);                      \
  }
#define KQ_MX_DEEP_STAGE(CUR, NXT, WAIT)                    \
  {                                                         \
    own_bytes(sa, sb);                                      \
    read_scales(CUR, 1, ta, tb);                            \
    read(CUR, 2, za, zb);                                   \
    read(CUR, 3, ua, ub);                                   \
    mma0(xa, xb, sa, sb);                                   \
    mma1(ya, yb, sa, sb);                                   \
    KQ_MX_SPREAD(2 * (MT + NT) + 2, 0)                      \
    WAIT;                                                   \
    __builtin_amdgcn_s_waitcnt(WAIT_LGKM0);                 \
    lds_barrier();                                          \
    own_bytes(ta, tb);                                      \
    issue(CUR);                                             \
    read_scales(NXT, 0, sa, sb);                            \
    read(NXT, 0, xa, xb);                                   \
    read(NXT, 1, ya, yb);                                   \
    mma0(za, zb, ta, tb);                                   \
    mma1(ua, ub, ta, tb);                                   \
    _Pragma("unroll") for (int i_ = 0; i_ < MT * NT; ++i_) { \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);    \
      __builtin_amdgcn_sched_group_barrier(0x020, (COPIES + MT * NT - 1) / (MT * NT), 1); \
      __builtin_amdgcn_sched_group_barrier(0x100, 3, 1);    \
    }                                                       \
    __builtin_amdgcn_sched_barrier(0);                      \
  }
  // Waits for the next stage's copies.  Newer than they are those of RING - 2 stages and, in the
  // first RING - 1 stages of a tile (`after`: there was one before), its 16 MT stores, which may stay
  // outstanding (the counter holds 63).  One block of instructions: a branch that the compiler sees
  // would let it move the matrix instructions across.
  constexpr int NEWER = (RING - 2) * COPIES, STORES = NEWER + 16 * MT < 63 ? NEWER + 16 * MT : 63;
  auto wait_stage = [&](bool after) {
    asm volatile("s_waitcnt vmcnt(%1)\n\ts_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lstage%=\n\ts_waitcnt vmcnt(%2)\n.Lstage%=:"
                 :: "s"(__builtin_amdgcn_readfirstlane((int)after)), "n"(STORES), "n"(NEWER) : "scc", "memory");
  };
  const int rounds = (stages + RING - 1) / RING;   // stages past the last multiply zeros
  bool stored = false;
  const int size = a.y_bf16 ? 2 : 4;

  for (;;) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int k = 0; k < NT; ++k) acc[m][k] = f32x16{};
    id += turns;
    const bool more = id < end;
    Tile nt = t;
    if (more) nt = at_id(id);
    if (ROWS != X_ROWS && more && a.index) {
      const int r = min(64 * (wave % MT) + lane, nt.last - 1 - nt.m0);
      copy_lds<4>(rsrc(a.index + nt.m0, (int)ALL), 4 * r, (uint8_t*)(next_index + 64 * (wave % MT)));
    }
    // the next tile's copies follow the last ones of this tile: those of its last round
    auto aim_next = [&]() {
      if (more) aim(nt, [&](int r) {
        const int x = read_lds(next_index + r);
        return a.index ? x : nt.m0 + r;
      });
    };
    for (int k = 0; k < rounds; ++k) {
      if (k == rounds - 1) {
        if (ROWS != X_ROWS && k == 0) {   // the index's copies have no earlier barrier behind them
          __builtin_amdgcn_s_waitcnt(wait_vm(0));
          lds_barrier();
        }
        aim_next();
      }
      const bool after = k == 0 && stored;
      if constexpr (RING == 4) {
        KQ_MX_DEEP_STAGE(b0, b1, wait_stage(after))
        KQ_MX_DEEP_STAGE(b1, b2, wait_stage(after))
        KQ_MX_DEEP_STAGE(b2, b3, wait_stage(after))
        KQ_MX_DEEP_STAGE(b3, b0, wait_stage(false))
      } else if constexpr (DEEP) {
        KQ_MX_DEEP_STAGE(b0, b1, wait_stage(after))
        KQ_MX_DEEP_STAGE(b1, b0, wait_stage(false))
      } else {
        KQ_MX_STAGE(b0, b1, wait_stage(after))
        KQ_MX_STAGE(b1, b0, wait_stage(false))
      }
    }
    stored = true;

    // Lane l32 holds NT neighbouring columns of 16 MT rows.  The descriptor ends with the tile's
    // last row, so stores of rows past it are dropped, and so are those of lanes whose columns
    // pass the last one.
    uint8_t* y0 = (uint8_t*)a.y + ((int64_t)t.m0 * a.ldy + t.n0) * size;
    const int rows = t.last - t.m0, n = t.n0 + (wc * 32 + l32) * NT;
    // Row m's sums, held in accumulation registers up to here: read out ahead of the branches
    // below, all of them at once, they would not fit.
    auto take = [&](int m, f32x16 (&v)[NT]) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        v[k] = acc[m][k];
        asm volatile("" : "+a"(v[k]));
      }
    };
    if (!a.y_far && (t.n0 + BN <= a.N || a.N % NT == 0)) {
      const int pitch = (int)a.ldy * size;
      const __amdgpu_buffer_rsrc_t ry = rsrc(y0, rows < BM ? rows * pitch : OOB);
      const int first = (wr * 32 * MT + q * 4 * MT) * pitch + (wc * 32 + l32) * NT * size;
      const int at = n + NT <= a.N ? first : OOB;
      auto store = [&](auto put) {
        int lane_at = at;
        asm volatile("" : "+v"(lane_at));   // offsets of the two types apart: shared ones spill
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x16 sums[NT];
          take(m, sums);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float v[NT];
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              v[k] = sums[k][j];
              asm("" : "+v"(v[k]));   // side by side in the other registers: there is none left of these
            }
            put(lane_at + (((j >> 2) * 8 + (j & 3)) * MT + m) * pitch, v);
          }
        }
      };
      if (a.y_bf16)
        store([&](int off, const float (&v)[NT]) { store_bf16<NT>(ry, off, v); });
      else
        store([&](int off, const float (&v)[NT]) { store_f32<NT>(ry, off, v); });
    } else {
      // a last column that ends inside a lane's, or rows too far apart for 32-bit offsets
      int part = q;
      asm volatile("" : "+v"(part));   // its addresses computed here, not ahead of the loop
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x16 sums[NT];
        take(m, sums);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int r = wr * 32 * MT + ((j >> 2) * 8 + part * 4 + (j & 3)) * MT + m;
          const int64_t at = r * a.ldy + n - t.n0;
          const int cols = r < rows ? (int)min((int64_t)NT, a.N - n) : 0;
#pragma unroll
          for (int k = 0; k < NT; ++k)
            if (k < cols) {
              if (a.y_bf16)
                ((uint16_t*)y0)[at + k] = to_bf16(sums[k][j]);
              else
                ((float*)y0)[at + k] = sums[k][j];
            }
        }
      }
      __builtin_amdgcn_s_waitcnt(wait_vm(0));   // fewer stores than the next round's waits count on
    }
    if (!more) break;
    t = nt;
  }
#undef KQ_MX_STAGE
#undef KQ_MX_DEEP_STAGE
#undef KQ_MX_SPREAD
  // the ring's trailing copies must land before its LDS is released
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
}

size_t code_bytes(int64_t rows, int64_t n) { return (size_t)rows * (size_t)(mx_pad(n) / 2); }
size_t scale_bytes(int64_t rows, int64_t n) { return (size_t)rows * (size_t)(mx_pad(n) / 32); }

// Whether an index can reach past the 32-bit offsets of the copies.
bool x_far(const ProductArgs& p) { return p.rows * p.pitch >= 0xffff0000ll; }

// Row tiles of BM rows: at most, over any offsets.
int64_t row_tiles(const ProductArgs& p, int bm) {
  return ceil_div(p.slots, bm) + (p.offsets ? std::min<int64_t>(p.experts, p.slots) : 0);
}

template <int MT, int NT, int WC, int RING>
kq_status launch_tiles(const ProductArgs& p, hipStream_t s) {
  constexpr int BM = 64 * MT, BN = 32 * NT * WC;
  // one workgroup for each place on the card, or for each tile if there are fewer
  constexpr int PLACES = 160 * 1024 / (RING * (BM + BN) * 136 + (1 << 13));
  const int64_t total = std::min<int64_t>(ceil_div(row_tiles(p, BM) * ceil_div(p.N, BN), 8),
                                          ceil_div(device_cu_count() * std::min(PLACES, 4), 8)) * 8;
  const dim3 grid((unsigned)total), block(128 * WC);
  if (!p.offsets)
    mx_tile_kernel<MT, NT, WC, RING, X_ROWS><<<grid, block, 0, s>>>(p);
  else if (!x_far(p))
    mx_tile_kernel<MT, NT, WC, RING, X_INDEX><<<grid, block, 0, s>>>(p);
  else if constexpr (MT == 4)
    mx_tile_kernel<MT, NT, WC, RING, X_FAR><<<grid, block, 0, s>>>(p);
  KQ_LAUNCHED("mx_tile_kernel");
  return KQ_OK;
}

// The tile with the least time.  Up to 64 rows (of an expert, on average) the layer's bytes are the
// bound, and the smallest tiles put the most workgroups at them: 8 experts of 11008 x 4096 and a
// token 14.2 us (64 x 128 tiles: 16.6), 64 of 1408 x 2048 and 96 tokens 19.6 (22.6).  With more
// rows, by a tile's time and the number of tiles that a compute unit gets: at K = 4096 and a full
// card 33 us for 256 x 256, 9.4 for 128 x 128, 4.5 for 64 x 64 (4096 x 4096 outputs: 39, 42 and 66
// in all; 2048 x 4096: 30, 24, 34; 256 x 4096: 24, 12, 8.6).  A smaller tile has to win clearly:
// its count rounds less, but it reads more.
kq_status launch_best(const ProductArgs& p, hipStream_t s) {
  static const struct { int id; double cost; } tiles[] = {{256, 33.0}, {128, 9.4}, {64, 4.5}};
  const int64_t active = p.offsets ? std::min<int64_t>(p.experts, p.slots) : 0;
  int64_t best = 64;
  if ((p.offsets ? ceil_div(p.slots, p.experts) : p.slots) > 64) {
    double least = 0;
    for (const auto& t : tiles) {
      // an expert's last tile is half full, on average, and it has one at least
      const int64_t tm = p.offsets ? std::max(active, p.slots / t.id + active / 2) : ceil_div(p.slots, t.id);
      const double cost = t.cost * (double)ceil_div(tm * ceil_div(p.N, t.id), device_cu_count());
      if (least == 0 || cost < 0.8 * least) {
        least = cost;
        best = t.id;
      }
    }
  }
  switch (p.offsets && x_far(p) ? 256 : testing_value(KQ_TESTING_MX_TILE, best)) {
    case 256: return launch_tiles<4, 2, 4, 2>(p, s);
    case 128: return launch_tiles<2, 2, 2, 2>(p, s);
    default: return launch_tiles<1, 1, 2, 4>(p, s);
  }
}

// Checks and quantises the activations (unless they are quantised already), then the product.
kq_status product(const char* fn, const MxRows& x, ProductArgs p, int y_type, void* ws, size_t ws_bytes,
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
    KQ_TRY(mx_check_rows(fn, x, &block));
    if (x.scales) return fail(KQ_EINVAL, "%s: scales go with quantised rows only", fn);
  }
  if (y_type != KQ_F32 && y_type != KQ_BF16) return fail(KQ_EINVAL, "%s: output type %d", fn, y_type);
  if (p.N < 1 || p.N > MX_MAX_N) return fail(KQ_ESHAPE, "%s: %lld output channels", fn, (long long)p.N);
  if (p.ldy < p.N) return fail(KQ_ESHAPE, "%s: ldy %lld < %lld", fn, (long long)p.ldy, (long long)p.N);
  if (!p.wc || !p.ws) return fail(KQ_EINVAL, "%s: NULL weights", fn);
  if (!aligned16(p.wc) || !aligned16(p.ws)) return fail(KQ_EINVAL, "%s: weights must be 16-byte aligned", fn);
  if (p.slots > 0 && !p.y) return fail(KQ_EINVAL, "%s: NULL output", fn);
  const int size = y_type == KQ_F32 ? 4 : 2;
  if ((uintptr_t)p.y & (size - 1)) return fail(KQ_EINVAL, "%s: output not aligned to its type", fn);
  p.pitch = mx_pad(x.n) / 2;
  p.steps = (int)(mx_pad(x.n) / MX_GROUP);
  p.rows = x.rows;
  p.y_bf16 = y_type == KQ_BF16;
  p.y_far = p.ldy > (1 << 20);
  if (x.type == KQ_MXFP4) {
    p.xc = (const uint8_t*)x.x;
    p.xs = x.scales;
  } else {
    const size_t need = code_bytes(x.rows, x.n) + scale_bytes(x.rows, x.n);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws)))
      return fail(KQ_EWORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    p.xc = (uint8_t*)ws;
    p.xs = (uint8_t*)ws + code_bytes(x.rows, x.n);
  }
  if (p.slots == 0) return KQ_OK;
  if (x.type != KQ_MXFP4 && mx_few_fused(p, x)) return mx_few_product(p, x, block, true, s);
  if (x.type != KQ_MXFP4) KQ_TRY(mx_quantize(x, block, (uint8_t*)p.xc, (uint8_t*)p.xs, nullptr, 0, s));
  if (mx_few(p)) return mx_few_product(p, x, block, false, s);
  return launch_best(p, s);
}

}  // namespace
}  // namespace kq

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
  return product("kq_mxfp4_linear", MxRows{x, x_type, rows, in, ldx, x_scales, d, sign, had}, p, y_type, ws,
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
  return product(fn, MxRows{x, x_type, rows, in, ldx, x_scales, d, sign, had}, p, y_type, ws, ws_bytes,
                 as_stream(stream));
}
