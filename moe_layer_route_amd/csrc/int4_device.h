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

// The masks of int4_operand in registers (v_and_or_b32 takes no literal; left
// to itself the compiler makes two instructions with one literal each).
struct Int4Masks {
  uint32_t field, base;
  __device__ __forceinline__ Int4Masks() {
    asm("v_mov_b32 %0, 0x00780078" : "=v"(field));
    asm("s_mov_b32 %0, 0x41804180" : "=s"(base));
  }
};

// codes of one word -> the bf16 operand 16 + q
__device__ __forceinline__ u32x4_t int4_operand(uint32_t w, const Int4Masks& m) {
  return u32x4_t{(w & m.field) | m.base, ((w >> 4) & m.field) | m.base, ((w >> 8) & m.field) | m.base,
                 (__builtin_amdgcn_alignbit(w, w, 12) & m.field) | m.base};
}

}  // namespace moe
