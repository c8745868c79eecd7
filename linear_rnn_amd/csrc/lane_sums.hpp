// Sums across the four rows of 16 lanes of a wave, shared by the linear attention and the layer norm.
#pragma once

#include "wkv7_device.hpp"

namespace rwkv7 {

// Sum over the lanes l, l ^ 16, l ^ 32, l ^ 48 (the same place of the four rows), the same bits in each: a swap
// of odd with even rows of two copies, then of the halves, leaves both partners' values in every lane.
__device__ __forceinline__ float pair_rows_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}
__device__ __forceinline__ float halves_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}
__device__ __forceinline__ float rows_sum(float x) { return halves_sum(pair_rows_sum(x)); }

}  // namespace rwkv7
