// Reductions over the lanes of a wave (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>

namespace kq {
namespace {

// The value of another lane of the same sixteen: part of the operation that takes it.
template <int CTRL, typename V>
__device__ __forceinline__ V moved(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// f over each LANES (16 or 64) lanes, the result in all of them: rotations inside sixteen, then
// exchanges of sixteens and of halves.
template <int LANES, typename V, typename F>
__device__ __forceinline__ V reduce_lanes(V v, F f) {
  v = f(v, moved<0x128>(v));
  v = f(v, moved<0x124>(v));
  v = f(v, moved<0x122>(v));
  v = f(v, moved<0x121>(v));
  if constexpr (LANES == 64) {
    unsigned u = __builtin_bit_cast(unsigned, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const unsigned a0 = a[0], a1 = a[1];
    v = f(__builtin_bit_cast(V, a0), __builtin_bit_cast(V, a1));
    u = __builtin_bit_cast(unsigned, v);
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned b0 = b[0], b1 = b[1];
    v = f(__builtin_bit_cast(V, b0), __builtin_bit_cast(V, b1));
  }
  return v;
}

}  // namespace
}  // namespace kq
