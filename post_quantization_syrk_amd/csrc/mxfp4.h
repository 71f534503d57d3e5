// What the MXFP4 sources share (not part of the C ABI): the held layout, launch arguments.
//
// A row of n values is held in blocks of 32: a scale 2^e per block and one E2M1 element per
// value.  With a the block's largest magnitude,
//   e = max(floor(log2 a) - 2, -127),   element = x / 2^e rounded to nearest, ties to even,
// on {0, 0.5, 1, 1.5, 2, 3, 4, 6}, magnitudes above 6 to 6.  A block with an infinity or a
// NaN has the scale byte 255, which every reader takes as NaN, and zero elements.
#pragma once

#include "device_util.h"
#include "kq_internal.h"

namespace kq {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int MX_BLOCK = 32;     // values per scale
constexpr int MX_GROUP = 128;    // columns per scale dword; rows are padded to whole groups
constexpr int64_t MX_MAX_ROWS = (int64_t)1 << 30, MX_MAX_N = (int64_t)1 << 24;

__host__ __device__ inline int64_t mx_pad(int64_t n) { return (n + MX_GROUP - 1) / MX_GROUP * MX_GROUP; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Activations of a call: rows to quantise (KQ_F32, KQ_BF16) or quantised rows (KQ_MXFP4).
struct MxRows {
  const void* x;
  int type;
  int64_t rows, n, ld;
  const uint8_t* scales;   // of quantised rows
  const float* d;
  const int8_t* sign;
  int64_t had;
};

// Checks rows that are to be quantised; *block: the Hadamard block.
kq_status mx_check_rows(const char* fn, const MxRows& r, int64_t* block);

// Enqueues the quantisation of checked rows.
kq_status mx_quantize(const MxRows& r, int64_t block, uint8_t* codes, uint8_t* scales, uint16_t* values,
                      int64_t ldv, hipStream_t s);

}  // namespace kq
