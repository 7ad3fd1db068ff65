// Device-side helpers of MXFP4: E2M1 codes and UE8M0 scales of rows.
#pragma once

#include "device_common.h"
#include "wave_reduce.h"

namespace moe {

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// UE8M0 byte -> float32 scale 2^(s - 127) (s = 0 is the subnormal 2^-127, 255 NaN)
__device__ __forceinline__ float ue8m0_to_f32(uint32_t s) {
  uint32_t u = s << 23;
  u = s == 0 ? 0x00400000u : u;
  u = s == 255 ? 0x7FC00000u : u;
  return __uint_as_float(u);
}

// eight E2M1 codes (one dword, k = 0..7 from the low nibble up) -> eight bf16 * scale
__device__ __forceinline__ u32x4_t dequant8(uint32_t w, float s) {
  const bf16x2_v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2_v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2_v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2_v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return u32x4_t{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                 __builtin_bit_cast(uint32_t, d)};
}

// The scale byte of a block whose largest |bf16| has these bits (a NaN's lie
// above infinity's): floor(log2 max) - 2 + 127, clamped at 0, where a zero or
// subnormal maximum lands too; 255 (NaN) for a block that is not finite.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t s = (uint32_t)max((int)(amax_bits >> 7) - 2, 0);
  return amax_bits >= 0x7F80u ? 255u : s;
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t pair) { return max(pair & 0x7FFFu, (pair >> 16) & 0x7FFFu); }

// two bf16 / scale -> two E2M1 codes in byte SEL of old: nearest, ties to the
// even code, |v| above 5 to 6 (v_cvt_scalef32_pk_fp4_bf16: the same codes as
// comparing with the midpoints, for every bf16)
template <int SEL>
__device__ __forceinline__ uint32_t encode2(uint32_t old, uint32_t pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_v, pair), scale, SEL);
}

// the maximum over a row of 16 lanes, in each of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, moved<kXor1>(v));
  v = max(v, moved<kXor2>(v));
  v = max(v, moved<kHalfMirror>(v));
  return max(v, moved<kMirror>(v));
}

// MXFP4 codes and scales of values 128 group .. of row r of a [R][K], by a row of 16
// lanes (this one is l): a quad of lanes has one block, the row one scale word.
// Whole rows of lanes call it.
__device__ __forceinline__ void quantize_128(const bf16_t* __restrict__ a, int64_t r, int64_t R, int K, int group,
                                             int l, uint32_t* __restrict__ codes, uint32_t* __restrict__ scales) {
  constexpr int kRowRor4 = 0x124, kRowRor8 = 0x128;   // rotations within a row of 16 lanes
  const int k = 128 * group + 8 * l;
  const bool in = r < R && k < K;
  u32x4_t v = u32x4_t{0u, 0u, 0u, 0u};
  if (in) v = ld16(a + r * K + k);
  uint32_t m = max(max(abs_max2(v.x), abs_max2(v.y)), max(abs_max2(v.z), abs_max2(v.w)));
  m = max(m, moved<kXor1>(m));
  m = max(m, moved<kXor2>(m));
  const uint32_t s = mx_scale_byte(m);
  const float scale = ue8m0_to_f32(s);
  uint32_t c = encode2<0>(0u, v.x, scale);
  c = encode2<1>(c, v.y, scale);
  c = encode2<2>(c, v.z, scale);
  c = encode2<3>(c, v.w, scale);
  if (s == 255) c = 0;
  if (in) codes[(r * K + k) / 8] = c;
  // the quads' scales, blocks past K 0, as one word
  uint32_t w = in ? s << (8 * (l / 4)) : 0u;
  w |= moved<kRowRor4>(w);
  w |= moved<kRowRor8>(w);
  if (l == 0 && r < R) scales[(int64_t)group * R + r] = w;
}

__device__ __forceinline__ i32x8_t fp4_operand(u32x4_t v) {
  return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}
// E2M1 x E2M1 products with block scales; OA, OB: which byte of a lane's scale
// word is its scale.  16x16x128: lane l holds row (column) l % 16 and the
// block l / 16 of 32 values; 32x32x64: row l % 32, block l / 32.
template <int OA, int OB>
__device__ __forceinline__ f32x4_t mfma_fp4_16(u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a), fp4_operand(b), c, 4, 4, OA, (int)sa, OB, (int)sb);
}
template <int OA, int OB>
__device__ __forceinline__ f32x16_t mfma_fp4_32(u32x4_t a, u32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(a), fp4_operand(b), c, 4, 4, OA, (int)sa, OB, (int)sb);
}

}  // namespace moe
