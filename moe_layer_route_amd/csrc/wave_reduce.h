// Reductions over a wave without LDS or lane permutations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Reductions over a wave by data-parallel moves: within quads, halves of rows
// and rows of 16 lanes (every lane of a row ends with the row's result, equal
// bits, since the operands of each step are symmetric), then the four rows.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ double add_moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return v + __builtin_bit_cast(double, (uint64_t)moved<CTRL>((uint32_t)(b >> 32)) << 32 | moved<CTRL>((uint32_t)b));
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_add(double v) {
  v = add_moved<kMirror>(add_moved<kHalfMirror>(add_moved<kXor2>(add_moved<kXor1>(v))));
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, moved<kXor1>(v));
  v = max(v, moved<kXor2>(v));
  v = max(v, moved<kHalfMirror>(v));
  v = max(v, moved<kMirror>(v));
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

template <int CTRL>
__device__ __forceinline__ uint64_t max_moved(uint64_t v) {
  const uint64_t o = (uint64_t)moved<CTRL>((uint32_t)(v >> 32)) << 32 | moved<CTRL>((uint32_t)v);
  return o > v ? o : v;
}
// the maximum over a row of 16 lanes, in each of them
__device__ __forceinline__ uint64_t row_max(uint64_t v) {
  return max_moved<kMirror>(max_moved<kHalfMirror>(max_moved<kXor2>(max_moved<kXor1>(v))));
}
__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  v = row_max(v);
  const uint64_t a = lane_u64(v, 0), b = lane_u64(v, 16), c = lane_u64(v, 32), d = lane_u64(v, 48);
  const uint64_t ab = a > b ? a : b, cd = c > d ? c : d;
  return ab > cd ? ab : cd;
}

}  // namespace moe
