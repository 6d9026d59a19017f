// Reductions over the 64 lanes of a wave.
#pragma once

#include "common.hpp"

namespace moelora {

// v of the lane that a DPP control names, `none` where there is none or its row of 16 lanes is
// not in ROWS
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp(T v, T none) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                             __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
  } else {
    const uint64_t a = __builtin_bit_cast(uint64_t, v), b = __builtin_bit_cast(uint64_t, none);
    const uint32_t lo = dpp<CTRL, ROWS>((uint32_t)a, (uint32_t)b);
    const uint32_t hi = dpp<CTRL, ROWS>((uint32_t)(a >> 32), (uint32_t)(b >> 32));
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  }
}

// f over all lanes of v, to every lane, in an order that does not change: within a row of 16 by
// shifts, then the rows.  (Exchanges through LDS wait for each other six times.)
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, T none, F&& f) {
  v = f(v, dpp<0x111, 0xF>(v, none));   // row_shr:1, 2, 4, 8
  v = f(v, dpp<0x112, 0xF>(v, none));
  v = f(v, dpp<0x114, 0xF>(v, none));
  v = f(v, dpp<0x118, 0xF>(v, none));
  v = f(v, dpp<0x142, 0xA>(v, none));   // row_bcast:15 to rows 1 and 3
  v = f(v, dpp<0x143, 0xC>(v, none));   // row_bcast:31 to rows 2 and 3
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
  } else {
    const uint64_t a = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)a, 63);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(a >> 32), 63);
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  }
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  return wave_reduce(v, T(0), [](T a, T b) { return a + b; });
}
// The same of fp64, whose additions cannot take another lane's number as they read it: it is moved first,
// and a 0 for a lane that is not there comes with the move.  (Rows that the others leave out add here what
// no one reads: lane 63 has the same sum, to the bit.)
template <int CTRL>
__device__ __forceinline__ double add_lane(double v) {
  const uint64_t a = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)a, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(a >> 32), CTRL, 0xF, 0xF, true);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <>
__device__ __forceinline__ double wave_sum(double v) {
  v = add_lane<0x143>(add_lane<0x142>(add_lane<0x118>(add_lane<0x114>(add_lane<0x112>(add_lane<0x111>(v))))));
  const uint64_t a = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)a, 63);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(a >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// of values none of which is below `none`
template <typename T>
__device__ __forceinline__ T wave_max(T v, T none) {
  return wave_reduce(v, none, [](T a, T b) { return a > b ? a : b; });
}
// of numbers (NaN would be lost as the first of a pair, and take the other's place as the second), as
// integers in the same order: their maximum takes another lane's in one instruction
__device__ __forceinline__ float wave_max(float v) {
  auto flip = [](int32_t b) { return b ^ (b >> 31 & 0x7FFFFFFF); };
  const int32_t none = INT32_MIN;
  return __builtin_bit_cast(float, flip(wave_max(flip(__builtin_bit_cast(int32_t, v)), none)));
}

}  // namespace moelora
