// Residual addition and RMS norm ahead of the block, with the normalised rows
// in bf16 (the router's and the bf16/4-bit experts' input) and, for the FP8
// experts, as E4M3 codes with one scale per row.
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 2 (the block runs on the
// normalised hidden state) and section 5 (FP8 activations with dynamic
// scales).  Per row t of H values:
//   r = bf16(x + residual)            (r = x without a residual)
//   inv = float32(1 / sqrt(sum_h r[h]^2 / H + eps)), the sum in float64: the
//         squares of bf16 values are exact there, so the result does not
//         depend on how a row is split over lanes, beyond the last bit of a
//         float64 sum
//   v = (r * inv) * gamma             (float32, each product rounded)
//   y = bf16(v)
//   s = max|v| / 448, code = E4M3(v * (448 / max|v|)): from the float32 values,
//         not from y, so a code carries one rounding and not two.  Below 2^-119,
//         where 448 / max|v| leaves float32, v and the maximum are taken times
//         2^64, which is exact.
//
// It is a stream: x and residual are read once, r, y and the codes written
// once, the row stays in registers between the two reductions.  T = 16384 rows
// of 2880 with a residual and codes (425 MB) take 75.6 us, 5.6 TB/s, which is
// what a large copy reaches (5.3 TB/s at 1 GB moved, 4.9 at 4 GB); one row
// takes 2.6 us.
#include "device_common.h"
#include "launch.h"
#include "wave_reduce.h"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr uint32_t kLiftBelow = 0x04000000u;   // bits of 2^-119
constexpr float kLift = 0x1p64f;

// E4M3 code of v, nearest with ties to even, saturated at 448, NaN -> 0x7F:
// with e = max(exponent, -6), q = rint(|v| * 2^(3-e)) counts quanta of
// 2^(e-3), and the code is (e + 6) * 8 + q (q = 16 carries into the next
// binade).  For rows whose scale is not an ordinary number.
__device__ __forceinline__ uint32_t e4m3_any(float v) {
  const uint32_t sign = (__float_as_uint(v) >> 24) & 0x80u;
  const float a = fminf(fabsf(v), kE4m3Max);
  const int e = max((int)(__float_as_uint(a) >> 23) - 127, -6);
  const uint32_t q = (uint32_t)__builtin_rintf(__builtin_amdgcn_ldexpf(a, 3 - e));
  const uint32_t code = sign | (uint32_t)((e + 6) * 8 + (int)q);
  return v != v ? 0x7Fu : code;
}

constexpr int kNormMaxWaves = 16;
constexpr int64_t kNormMaxGrid = (int64_t)1 << 21;

// One row per workgroup at a time (the grid is cut at kNormMaxGrid rows: a
// launch holds fewer than 2^32 threads); thread i holds the 16-byte pieces i,
// i + blockDim, ... (P of them).  x, residual, residual_out and y carry no __restrict__: an
// output may be the very buffer of an input, and a thread reads all its
// pieces before it writes any.
template <int P, bool RES, bool FP8>
__global__ __launch_bounds__(kNormMaxWaves * kWave) void add_rmsnorm_kernel(
    const bf16_t* x, const bf16_t* residual, const bf16_t* __restrict__ gamma, int T, int H, double eps,
    bf16_t* residual_out,
    bf16_t* y, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  // two of each: a wave may begin the next row while another still reads
  __shared__ double s_sum[2][kNormMaxWaves];
  __shared__ uint32_t s_max[2][kNormMaxWaves];
  const int np = H / 8;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int wave = tid / kWave, lane = tid & (kWave - 1), waves = nt / kWave;
  const u32x4_t zero = u32x4_t{0u, 0u, 0u, 0u};

  int parity = 1;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x) {
    parity ^= 1;
    const size_t base = (size_t)row * (size_t)H;

    u32x4_t r[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int i = tid + p * nt;
      r[p] = i < np ? *reinterpret_cast<const u32x4_t*>(x + base + 8 * (size_t)i) : zero;
    }
    if (RES) {
      u32x4_t a[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int i = tid + p * nt;
        a[p] = i < np ? *reinterpret_cast<const u32x4_t*>(residual + base + 8 * (size_t)i) : zero;
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          r[p][q] = pack_bf16x2(bf16lo(r[p][q]) + bf16lo(a[p][q]), bf16hi(r[p][q]) + bf16hi(a[p][q]));
    }
    u32x4_t gm[P];   // asked for ahead of the reduction, used behind it
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int i = tid + p * nt;
      gm[p] = i < np ? *reinterpret_cast<const u32x4_t*>(gamma + 8 * (size_t)i) : zero;
    }
    double ss = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const double lo = bf16lo(r[p][q]), hi = bf16hi(r[p][q]);
        ss = __builtin_fma(lo, lo, ss);
        ss = __builtin_fma(hi, hi, ss);
      }
    ss = wave_add(ss);
    if (waves > 1) {
      if (lane == 0) s_sum[parity][wave] = ss;
      __syncthreads();
      ss = 0.0;
      for (int w = 0; w < waves; ++w) ss += s_sum[parity][w];
    }
    const float inv = (float)(1.0 / sqrt(ss / (double)H + eps));

    float v[P][8];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int i = tid + p * nt;
      const u32x4_t g = gm[p];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[p][2 * q] = (bf16lo(r[p][q]) * inv) * bf16lo(g[q]);
        v[p][2 * q + 1] = (bf16hi(r[p][q]) * inv) * bf16hi(g[q]);
      }
      if (i < np) {
        if (RES) *reinterpret_cast<u32x4_t*>(residual_out + base + 8 * (size_t)i) = r[p];
        if (!FP8 || y != nullptr)
          *reinterpret_cast<u32x4_t*>(y + base + 8 * (size_t)i) =
              u32x4_t{pack_bf16x2(v[p][0], v[p][1]), pack_bf16x2(v[p][2], v[p][3]), pack_bf16x2(v[p][4], v[p][5]),
                      pack_bf16x2(v[p][6], v[p][7])};
        // the maximum on the bit patterns: a NaN compares above every number
        if (FP8)
#pragma unroll
          for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[p][q]) & 0x7FFFFFFFu);
      }
    }
    if (!FP8) continue;
    m = wave_max(m);
    if (waves > 1) {
      if (lane == 0) s_max[parity][wave] = m;
      __syncthreads();
      m = 0;
      for (int w = 0; w < waves; ++w) m = max(m, s_max[parity][w]);
    }
    const float amax = __uint_as_float(m);
    const float s = m == 0 ? 1.0f : __fdiv_rn(amax, kE4m3Max);
    const float lift = m < kLiftBelow ? kLift : 1.0f;
    const float up = m == 0 ? 1.0f : __fdiv_rn(kE4m3Max, amax * lift);
    // From 2^-119 on nothing is lifted, and |v * up| rounds to 448 at most:
    // the conversion instruction (nearest, ties to even) never overflows.
    const bool ordinary = __builtin_amdgcn_readfirstlane(m) - kLiftBelow < 0x7F800000u - kLiftBelow;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int i = tid + p * nt;
      u32x2_t c;
      if (ordinary) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[p][4 * h] * up, v[p][4 * h + 1] * up, 0, false);
          c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[p][4 * h + 2] * up, v[p][4 * h + 3] * up, w, true);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          c[h] = e4m3_any(v[p][4 * h] * lift * up) | e4m3_any(v[p][4 * h + 1] * lift * up) << 8 |
                 e4m3_any(v[p][4 * h + 2] * lift * up) << 16 | e4m3_any(v[p][4 * h + 3] * lift * up) << 24;
      }
      if (i < np) *reinterpret_cast<u32x2_t*>(codes + base + 8 * (size_t)i) = c;
    }
    if (tid == 0) scales[row] = s;
  }
}

template <int P>
hipError_t launch_p(const void* x, const void* residual, const void* gamma, int64_t T, int H, float eps,
                    void* residual_out, void* y, void* codes, float* scales, hipStream_t stream) {
  const int np = H / 8;
  const int waves = (np + kWave * P - 1) / (kWave * P);
  auto kern = residual ? (codes ? add_rmsnorm_kernel<P, true, true> : add_rmsnorm_kernel<P, true, false>)
                       : (codes ? add_rmsnorm_kernel<P, false, true> : add_rmsnorm_kernel<P, false, false>);
  const int64_t grid = T < kNormMaxGrid ? T : kNormMaxGrid;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(waves * kWave), 0, stream, (const bf16_t*)x,
                     (const bf16_t*)residual, (const bf16_t*)gamma, (int)T, H, (double)eps,
                     (bf16_t*)residual_out, (bf16_t*)y, (uint8_t*)codes, scales);
  return hipGetLastError();
}

}  // namespace

// Two pieces a thread: at H = 2880 (three waves a row) T = 64 takes 3.5 us and
// T = 16384 75.6 us, against 4.0 and 76.2 with one piece (six waves) and 5.4
// and 82.9 with four (two waves; that one with reductions by lane permutations,
// which the moves of wave_reduce.h have replaced).  Rows that one wave
// covers with one piece a thread take that: 8192 x 512 9.1 against 10.1 us.
// H <= 16384 is 2048 pieces: at most 16 waves a row.
hipError_t launch_add_rmsnorm(const void* x, const void* residual, const void* gamma, int64_t T, int H, float eps,
                              void* residual_out, void* y, void* codes, float* scales, hipStream_t stream) {
  if (H / 8 <= kWave) return launch_p<1>(x, residual, gamma, T, H, eps, residual_out, y, codes, scales, stream);
  return launch_p<2>(x, residual, gamma, T, H, eps, residual_out, y, codes, scales, stream);
}

}  // namespace moe
