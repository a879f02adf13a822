// wave_ops.hpp -- sums and maxima over the lanes of a wave, on the vector ALU.
#pragma once

#include "mm_device.hpp"

namespace mmk {

// The largest of a wave's values, and their sum, for all lanes: six steps of the vector ALU (within
// rows of 16 lanes, then across them) and not six exchanges through LDS, each of which waits for the
// one before.  Lanes with no neighbour to take from meet 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_take(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, lane_take<0x111, 0xf>(v));
  v = max(v, lane_take<0x112, 0xf>(v));
  v = max(v, lane_take<0x114, 0xf>(v));
  v = max(v, lane_take<0x118, 0xf>(v));
  v = max(v, lane_take<0x142, 0xa>(v));
  v = max(v, lane_take<0x143, 0xc>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float lane_add(float v) {
  return v + __builtin_bit_cast(float, lane_take<CTRL, ROWS>(__builtin_bit_cast(uint32_t, v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = lane_add<0x111, 0xf>(v);
  v = lane_add<0x112, 0xf>(v);
  v = lane_add<0x114, 0xf>(v);
  v = lane_add<0x118, 0xf>(v);
  v = lane_add<0x142, 0xa>(v);
  v = lane_add<0x143, 0xc>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// A lane's value and those of the lanes of its row of 16 at the same place in their runs of N
// (4 or 8) lanes.
template <int N>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (N == 4) v = lane_add<0x124, 0xf>(v);
  return lane_add<0x128, 0xf>(v);
}

}  // namespace mmk
