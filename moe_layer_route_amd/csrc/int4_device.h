// Shared by the int4 kernels: the weight tiles and their operands.
#pragma once

#include "device_common.h"

namespace moe {

constexpr int kTileN = 64, kTileK = 32, kTileBytes = 1024;

typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// A lane's offset and the wave's: no address arithmetic per load.
template <int AUX = 0>
__device__ __forceinline__ u32x4_t buf_ld16(rsrc_t r, uint32_t lane_off, uint32_t wave_off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)lane_off, (int)wave_off, AUX));
}

// codes of one word -> the bf16 operand 16 + q
__device__ __forceinline__ u32x4_t int4_operand(uint32_t w) {
  const uint32_t m = 0x00780078u, o = 0x41804180u;
  return u32x4_t{(w & m) | o, ((w >> 4) & m) | o, ((w >> 8) & m) | o,
                 (__builtin_amdgcn_alignbit(w, w, 12) & m) | o};
}

}  // namespace moe
