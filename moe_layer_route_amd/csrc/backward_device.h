// Sums of the block's backward pass that run beside its products (backward_gemm.hip)
// and beside the sum of the input gradients (backward.hip).
#pragma once
#include "device_common.h"
#include "launch.h"

namespace moe {
namespace {

#define LDS3 __attribute__((address_space(3)))

// 16 bytes of a bias or of its gradient, which need not begin at more than a word
typedef u32x4_t u32x4_word_t __attribute__((aligned(4)));

// the permutation's arrays, as permute.hip leaves them
struct Permuted {
  const int32_t *cnt, *off, *rows;
  uint32_t per_token;   // slot / k = umulhi(slot, per_token); 0: k = 1
};

__device__ __forceinline__ uint32_t token_of(uint32_t slot, uint32_t per_token) {
  return per_token ? __umulhi(slot, per_token) : slot;
}

// slot / k for the slots that can be (T H below 2^30 and H >= 8: below 2^30) as the
// high word of slot times 2^32 / k rounded up: off by less than slot / 2^30 / k
inline uint32_t per_token(int k) { return k == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + k - 1) / k); }

// ---------------------------------------------------------------------------
// Column sums over an expert's slots, of rows V[..] times a factor of the slot: dbgu
// sums dgu, dbd w dy, dWr dl x and dbr dl.  One workgroup per expert and 512
// columns, its four waves take every fourth row, eight columns a lane, eight rows in
// flight; the sums meet in LDS in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kSumWaves = 4;
constexpr int kSumAhead = 8;
constexpr int kSumCols = 8 * kWave;
constexpr int kSumLds = kSumWaves * (8 * kWave + 1) * 4;

struct Sum {
  const bf16_t* V;
  const float* factor;   // of the slot; null: 1, and V has the rows of the permuted order, else the tokens'
  int C, parts;          // columns, pieces of 512 of them (0: not asked for)
  bf16_t *out, *out_factor;   // [E][C]; [E], the sum of the factors, or null
};

template <bool GATHER>
__device__ __forceinline__ void column_sum(const Sum& p, const Permuted& a, int e, int piece, LDS3 char* smem) {
  LDS3 float (*part)[8][kWave] = (LDS3 float (*)[8][kWave])smem;
  LDS3 float* part_f = (LDS3 float*)(smem + kSumWaves * 8 * kWave * 4);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n = a.cnt[e], row0 = a.off[e], C = p.C;
  const int col = piece * kSumCols + 8 * lane;
  const int at = min(col, C - 8);   // C % 8 == 0
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum_f = 0.f;
  for (int m0 = wave; m0 < n; m0 += kSumWaves * kSumAhead) {
    u32x4_t v[kSumAhead];
    float f[kSumAhead];
#pragma unroll
    for (int i = 0; i < kSumAhead; ++i) {
      const int at_m = row0 + min(m0 + kSumWaves * i, n - 1);
      const uint32_t slot = GATHER ? (uint32_t)a.rows[at_m] : 0u;
      const size_t row = GATHER ? token_of(slot, a.per_token) : (size_t)at_m;
      f[i] = GATHER ? p.factor[slot] : 1.f;
      v[i] = ld16(p.V + row * C + at);
    }
#pragma unroll
    for (int i = 0; i < kSumAhead; ++i) {
      if (m0 + kSumWaves * i < n) {   // wave-uniform
        sum_f += f[i];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum[2 * q] = fmaf(f[i], bf16lo(v[i][q]), sum[2 * q]);
          sum[2 * q + 1] = fmaf(f[i], bf16hi(v[i][q]), sum[2 * q + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) part[wave][q][lane] = sum[q];
  if (lane == 0) part_f[wave] = sum_f;
  __syncthreads();
  if (wave == 0) {
    float s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      s[q] = part[0][q][lane];
#pragma unroll
      for (int w = 1; w < kSumWaves; ++w) s[q] += part[w][q][lane];
    }
    if (col < C)
      *reinterpret_cast<u32x4_word_t*>(p.out + (size_t)e * C + col) =
          u32x4_t{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7])};
    if (p.out_factor && piece == 0 && lane == 0) {
      float f = part_f[0];
#pragma unroll
      for (int w = 1; w < kSumWaves; ++w) f += part_f[w];
      p.out_factor[e] = (bf16_t)f32_to_bf16(f);
    }
  }
}

inline Sum sum_of(const void* V, const float* factor, int C, void* out, void* out_factor) {
  return Sum{(const bf16_t*)V, factor, C, out ? (C + kSumCols - 1) / kSumCols : 0, (bf16_t*)out, (bf16_t*)out_factor};
}

// ---------------------------------------------------------------------------
// dw and dl of token t by one wave; its lanes split the columns of dy and bd, and
// the parts of the sums over i that the products left.
// ---------------------------------------------------------------------------
struct Dl {
  const bf16_t *dy, *bd;
  const int32_t *ids, *pos;
  const float *w, *dw_part;   // [T][k]; [parts][S]
  int parts, H, k;
  int64_t T;
  float* dl;                  // [T][k]
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

__device__ __forceinline__ void token_dl(const Dl& p, int64_t t, int lane) {
  const int k = p.k, H = p.H;
  const int64_t S = p.T * k;
  // a skipped slot's weight takes no part, whatever it is
  float dw[MOE_MAX_K_DEV], w[MOE_MAX_K_DEV];
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j) {
    dw[j] = w[j] = 0.f;
    if (j < k) {
      const int64_t s = t * k + j;
      const int at = p.pos[s];
      if (at >= 0) {   // wave-uniform
        float sum = 0.f;
        const u32x4_t* a = reinterpret_cast<const u32x4_t*>(p.dy + t * H);
        const u32x4_word_t* b = reinterpret_cast<const u32x4_word_t*>(p.bd + (size_t)p.ids[s] * H);
        for (int c = lane; c < H / 8; c += kWave) {
          const u32x4_t u = a[c], v = b[c];
#pragma unroll
          for (int q = 0; q < 4; ++q) sum = fmaf(bf16hi(u[q]), bf16hi(v[q]), fmaf(bf16lo(u[q]), bf16lo(v[q]), sum));
        }
        for (int q = lane; q < p.parts; q += kWave) sum += p.dw_part[(size_t)q * S + at];
        dw[j] = wave_sum(sum);
        w[j] = p.w[s];
      }
    }
  }
  float mean = 0.f;
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j)
    if (j < k) mean = fmaf(w[j], dw[j], mean);
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j)
    if (j < k && lane == j) p.dl[t * k + j] = w[j] * (dw[j] - mean);
}

}  // namespace
}  // namespace moe

#undef LDS3
