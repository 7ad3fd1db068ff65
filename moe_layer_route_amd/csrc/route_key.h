// The router's order of experts: by (float32 logit descending, index ascending).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Monotone map of float32 to uint32 (larger float -> larger key); -0 == +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t make_key(float v, int e) {
  return ((uint64_t)order_key(v) << 32) | (uint64_t)(0xFFFFu - (uint32_t)e);
}
__device__ __forceinline__ int key_expert(uint64_t k) { return (int)(0xFFFFu - (uint32_t)(k & 0xFFFFu)); }

}  // namespace moe
