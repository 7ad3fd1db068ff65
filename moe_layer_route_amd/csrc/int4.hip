// Expert weights as uniform 4-bit integers with group scales (W4A16): the
// quantiser, the packer, and the expert products.
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 5 (4-bit expert weights,
// bf16 activations) and section 2 (per-expert gate_up -> bias -> GLU, down ->
// bias).  A weight is (q - z) * s: q a code 0..15, s a bf16 scale and z a zero
// point (8 without zero points) for each group of G values of K in a column.
//
// Layout (K = contraction dimension, N = output columns):
//   codes  uint8 [E][ceil(N/64)][K/32][1024]: a tile holds 64 columns x 32
//          values of K as 64 lanes x four 32-bit words; word j of lane
//          16 g + c holds column 64 nt + 4 c + j, K = 32 kt + 8 g + i for
//          i = 0..7, with value i at bit (3 + 4 (i / 2) + 16 (i % 2)) mod 32.
//          A wave reads a tile as one contiguous kilobyte, 16 bytes a lane,
//          and a word turns into an MFMA operand without any exchange between
//          lanes: (rotate(word, 4 p) & 0x00780078) | 0x41804180 is the bf16
//          pair (16 + q[2p], 16 + q[2p + 1]).  Columns past N hold anything.
//   scales bf16 [E][ceil(K/G)][N], zeros uint8 of the same shape.
#include "device_common.h"
#include "launch.h"

namespace moe {
namespace {

constexpr int kTileN = 64, kTileK = 32, kTileBytes = 1024;

// bit of value i in its word
__device__ __forceinline__ int int4_bit(int i) { return (3 + 4 * (i >> 1) + 16 * (i & 1)) & 31; }
// eight codes, value i in bits 4i .. 4i+3, to the stored order
__device__ __forceinline__ uint32_t int4_store_order(uint32_t w) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t q = (w >> (4 * i)) & 15u;
    const int at = int4_bit(i);
    o |= q << at;
    if (at > 28) o |= q >> (32 - at);
  }
  return o;
}
__device__ __forceinline__ uint32_t int4_value(uint32_t w, int i) {
  const int at = int4_bit(i);
  return (at ? (w >> at) | (w << (32 - at)) : w) & 15u;
}

// ---------------------------------------------------------------------------
// Quantiser: one thread per (column, group).  Symmetric: s = bf16(max|v| / 7),
// q = clamp(rint(v / s), -8, 7) + 8.  With zero points: lo = min(v, 0),
// hi = max(v, 0), s = bf16(hi / 15 - lo / 15), z = clamp(rint(-lo / s), 0,
// 15), q = clamp(rint(v / s) + z, 0, 15).  float32, halves to even; s = 0
// gives q = z (and z = 0 with zero points).
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;

__global__ __launch_bounds__(kQThreads) void int4_quantize_kernel(const bf16_t* __restrict__ W, int K, int N, int G,
                                                                  uint32_t* __restrict__ codes,
                                                                  uint16_t* __restrict__ scales,
                                                                  uint8_t* __restrict__ zeros) {
  const int nt_n = (N + kTileN - 1) / kTileN;
  const int n = blockIdx.x * kQThreads + threadIdx.x;
  if (n >= nt_n * kTileN) return;   // no barrier in this kernel
  const int b = blockIdx.y, e = blockIdx.z;
  const int k0 = b * G, k1 = min(K, k0 + G);
  const bool in = n < N;
  const bf16_t* src = W + (size_t)e * K * N + n;
  float lo = 0.f, hi = 0.f;
  if (in)
    for (int k = k0; k < k1; ++k) {
      const float v = bf16_to_f32(src[(size_t)k * N]);
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
  lo = fabsf(lo);   // a zero takes no sign
  hi = fabsf(hi);
  const float want = zeros ? __fdiv_rn(hi, 15.0f) + __fdiv_rn(lo, 15.0f) : __fdiv_rn(fmaxf(hi, lo), 7.0f);
  const uint32_t sb = f32_to_bf16(want);
  const float s = bf16_to_f32(sb);
  float z = 8.0f;
  if (zeros) z = s == 0.0f ? 0.0f : fminf(fmaxf(__builtin_rintf(__fdiv_rn(lo, s)), 0.0f), 15.0f);
  if (in) {
    const size_t at = ((size_t)e * gridDim.y + b) * N + n;
    scales[at] = (uint16_t)sb;
    if (zeros) zeros[at] = (uint8_t)z;
  }
  const int c = (n % kTileN) / 4, j = n % 4;
  for (int k = k0; k < k1; k += 8) {
    uint32_t w = 0;
    if (in)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = bf16_to_f32(src[(size_t)(k + i) * N]);
        const float q = s == 0.0f ? z : fminf(fmaxf(__builtin_rintf(__fdiv_rn(v, s)) + z, 0.0f), 15.0f);
        w |= (uint32_t)q << (4 * i);
      }
    const int kt = k / kTileK, g = (k % kTileK) / 8;
    codes[(((size_t)e * nt_n + n / kTileN) * (K / kTileK) + kt) * (kTileBytes / 4) + (16 * g + c) * 4 + j] =
        int4_store_order(w);
  }
}

// Codes [E][N][K/2] (K contiguous, low nibble first) to the tile order: one
// thread per stored word, which is four consecutive source bytes.
__global__ __launch_bounds__(kQThreads) void int4_pack_kernel(const uint8_t* __restrict__ src, int K, int N,
                                                              uint32_t* __restrict__ codes) {
  const int nt_n = (N + kTileN - 1) / kTileN;
  const int word = threadIdx.x;                     // 256 words a tile
  const int kt = blockIdx.x, e = blockIdx.z;
  const int lane = word / 4, g = lane / 16, c = lane % 16, j = word % 4;
  for (int nt = blockIdx.y; nt < nt_n; nt += gridDim.y) {
    const int n = nt * kTileN + 4 * c + j;
    const uint32_t w =
        n < N ? *reinterpret_cast<const uint32_t*>(src + ((size_t)e * N + n) * (K / 2) + 16 * (size_t)kt + 4 * g) : 0u;
    codes[(((size_t)e * nt_n + nt) * (K / kTileK) + kt) * (kTileBytes / 4) + word] = int4_store_order(w);
  }
}

// ---------------------------------------------------------------------------
// Expert products: one wave per (expert, 64 columns), a lane per column, four
// token rows at a time.  Group sums of (q - z) * a in float32, scaled once per
// group.
// ---------------------------------------------------------------------------
template <bool GATE_UP>
__global__ __launch_bounds__(kWave) void int4_kernel(const bf16_t* __restrict__ A, const uint32_t* __restrict__ Wq,
                                                     const uint16_t* __restrict__ Ws, const uint8_t* __restrict__ Wz,
                                                     const bf16_t* __restrict__ bias, const int32_t* __restrict__ cnt,
                                                     const int32_t* __restrict__ off, const int32_t* __restrict__ rows,
                                                     int K, int N, int G, int kslots, void* __restrict__ out) {
  const int e = blockIdx.y, M = cnt[e];
  if (M == 0) return;
  const int row0 = off[e];
  const int lane = threadIdx.x, c = lane / 4, j = lane % 4;
  const int n = blockIdx.x * kTileN + lane;
  const int nc = min(n, N - 1);
  const int ng = (K + G - 1) / G, nkt = K / kTileK;
  const uint32_t* wp = Wq + ((size_t)e * gridDim.x + blockIdx.x) * (size_t)nkt * (kTileBytes / 4) + c * 4 + j;
  for (int r0 = 0; r0 < M; r0 += 4) {
    const bf16_t* ap[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int r = row0 + min(r0 + m, M - 1);
      ap[m] = A + (size_t)(GATE_UP ? rows[r] / kslots : r) * K;
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < ng; ++b) {
      const size_t at = ((size_t)e * ng + b) * N + nc;
      const float s = bf16_to_f32(Ws[at]);
      const float z = Wz ? (float)Wz[at] : 8.0f;
      float part[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = b * G; k < min(K, (b + 1) * G); k += 8) {
        const uint32_t w = wp[(size_t)(k / kTileK) * (kTileBytes / 4) + (k % kTileK) * 8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = (float)int4_value(w, i) - z;
#pragma unroll
          for (int m = 0; m < 4; ++m) part[m] = __builtin_fmaf(bf16_to_f32(ap[m][k + i]), q, part[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = __builtin_fmaf(part[m], s, acc[m]);
    }
    const float bb = bf16_to_f32(bias[(size_t)e * N + nc]);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float v = acc[m] + bb;
      const float other = __shfl_xor(v, 1, kWave);
      if (r0 + m < M && n < N) {
        const size_t r = (size_t)(row0 + r0 + m);
        if (!GATE_UP)
          reinterpret_cast<float*>(out)[r * N + n] = v;
        else if (lane % 2 == 0)
          reinterpret_cast<uint16_t*>(out)[r * (N / 2) + n / 2] = (uint16_t)f32_to_bf16(clamped_glu(v, other));
      }
    }
  }
}

}  // namespace

hipError_t launch_int4_quantize(const void* W, int E, int K, int N, int G, void* codes, void* scales, void* zeros,
                                hipStream_t stream) {
  const int cols = (N + kTileN - 1) / kTileN * kTileN;
  dim3 grid((unsigned)((cols + kQThreads - 1) / kQThreads), (unsigned)((K + G - 1) / G), (unsigned)E);
  hipLaunchKernelGGL(int4_quantize_kernel, grid, dim3(kQThreads), 0, stream, (const bf16_t*)W, K, N, G,
                     (uint32_t*)codes, (uint16_t*)scales, (uint8_t*)zeros);
  return hipGetLastError();
}

hipError_t launch_int4_pack(const void* src, int E, int K, int N, void* codes, hipStream_t stream) {
  dim3 grid((unsigned)(K / kTileK), (unsigned)((N + kTileN - 1) / kTileN), (unsigned)E);
  hipLaunchKernelGGL(int4_pack_kernel, grid, dim3(kQThreads), 0, stream, (const uint8_t*)src, K, N, (uint32_t*)codes);
  return hipGetLastError();
}

hipError_t launch_int4_gate_up(const void* x, const void* Wq, const void* Ws, const void* Wz, const void* bgu,
                               const int32_t* cnt, const int32_t* off, const int32_t* rows, int H, int E, int k, int I,
                               int G, void* h, hipStream_t stream) {
  dim3 grid((unsigned)((2 * I + kTileN - 1) / kTileN), (unsigned)E);
  hipLaunchKernelGGL(int4_kernel<true>, grid, dim3(kWave), 0, stream, (const bf16_t*)x, (const uint32_t*)Wq,
                     (const uint16_t*)Ws, (const uint8_t*)Wz, (const bf16_t*)bgu, cnt, off, rows, H, 2 * I, G, k, h);
  return hipGetLastError();
}

hipError_t launch_int4_down(const void* h, const void* Wq, const void* Ws, const void* Wz, const void* bd,
                            const int32_t* cnt, const int32_t* off, int H, int E, int I, int G, float* o,
                            hipStream_t stream) {
  dim3 grid((unsigned)((H + kTileN - 1) / kTileN), (unsigned)E);
  hipLaunchKernelGGL(int4_kernel<false>, grid, dim3(kWave), 0, stream, (const bf16_t*)h, (const uint32_t*)Wq,
                     (const uint16_t*)Ws, (const uint8_t*)Wz, (const bf16_t*)bd, cnt, off, nullptr, I, H, G, 1, o);
  return hipGetLastError();
}

}  // namespace moe
