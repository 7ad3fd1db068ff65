// Grouped GEMMs of the experts with 4-bit integer weights (many rows per
// expert).
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 5 (one batched launch for
// all experts, 4-bit weights) and section 2 (gate_up -> bias -> GLU, down ->
// bias).  The format and the exact 16 + q operands are those of int4.hip.
//
// A workgroup owns 128 rows x 512 columns of one expert: eight waves, two per
// SIMD, each with a strip of 64 columns (128 accumulators a lane) and all 128
// rows.  K goes in units of GU tiles that never cross a group of the scales
// (64 values, or 32 where the groups are of 32).  A unit's token rows come into
// LDS by direct loads, fragment by fragment (a fragment is the 16-row operand
// of one MFMA, a kilobyte), three units ahead in a ring of four; its weights,
// two tiles a wave, straight into registers.  Per 16-row chunk the unit's
// products go into a fresh accumulator that starts at -(16 + z) sum(a) and is
// added to the result, times the scale, in float32.
#include "device_common.h"
#include "int4_device.h"
#include "launch.h"

namespace moe {
namespace {

constexpr int kGemmWaves = 8;
constexpr int kBM = 128, kChunks = kBM / 16;
constexpr int kBN = kGemmWaves * kTileN;
constexpr int kRing = 4;
constexpr int kXcds = 8;
constexpr int kMBlock = 8;   // M tiles per block of the tile order
constexpr uint32_t kOutOfRange = 0xFFFFFFF0u;

template <bool GATE_UP, int GU, bool ZERO>
__global__ __launch_bounds__(kGemmWaves * kWave, 2) void int4_gemm_kernel(
    const bf16_t* __restrict__ A, const uint8_t* __restrict__ Wq, const uint16_t* __restrict__ Ws,
    const uint8_t* __restrict__ Wz, const bf16_t* __restrict__ bias, const int32_t* __restrict__ cnt,
    const int32_t* __restrict__ off, const int32_t* __restrict__ rows, int K, int N, int E, int kslots, int64_t a_rows,
    int n_tiles, int units_per_group, void* __restrict__ out) {
  __shared__ __align__(16) u32x4_t lds[kRing][GU][kChunks][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int e, m0, nt;
  if (!grouped_gemm_tile(cnt, E, kBM, n_tiles, kMBlock, lane, e, m0, nt)) return;   // block-uniform
  const int M = cnt[e], row0 = off[e];
  const int nch = min(kChunks, (M - m0 + 15) / 16);   // chunks with rows
  const int g = lane >> 4, c = lane & 15;
  const int nkt = K / kTileK, nu = (nkt + GU - 1) / GU;
  const int ng = (nu + units_per_group - 1) / units_per_group;
  const int strips = (N + kTileN - 1) / kTileN;
  const int strip = nt * kGemmWaves + wave;
  const bool live = strip < strips;   // wave-uniform; a wave past the last strip only loads rows
  const int ncol = strip * kTileN + 4 * c;
  const uint32_t s_col = (uint32_t)min(ncol, N - 4);

  const rsrc_t w_rs = make_rsrc(Wq + ((size_t)e * strips + min(strip, strips - 1)) * (size_t)nkt * kTileBytes,
                                (uint32_t)nkt * kTileBytes);
  const rsrc_t s_rs = make_rsrc(Ws + (size_t)e * ng * N, (uint32_t)ng * N * 2);
  const rsrc_t z_rs = make_rsrc(ZERO ? Wz + (size_t)e * ng * N : Wq, ZERO ? (uint32_t)ng * N : 0u);
  const u32x4_t a_rs = rsrc_words(GATE_UP ? A : A + (size_t)row0 * K, (uint32_t)((size_t)(GATE_UP ? a_rows : M) * K * 2));

  // wave w brings in chunk w's fragments: lane (row c, group g)
  const int r = min(m0 + 16 * wave + c, M - 1);
  const uint32_t a_off = ((uint32_t)(GATE_UP ? rows[row0 + r] / kslots : r) * (uint32_t)K + 8u * g) * 2u;
  const uint32_t lds0 = (uint32_t)(uintptr_t)&lds[0][0][0][0];
  auto load_rows = [&](int u) {
    if (wave < nch) {
#pragma unroll
      for (int t = 0; t < GU; ++t) {
        const int kt = GU * u + t;
        dma16(a_rs, kt < nkt ? a_off : kOutOfRange, kt < nkt ? 64u * (uint32_t)kt : 0u,
              lds0 + (uint32_t)((((u % kRing) * GU + t) * kChunks + wave) * kWave) * 16u);
      }
    }
  };
  struct Unit {
    u32x4_t w[GU];
    u32x2_t s;
    uint32_t z;
  };
  auto load_weights = [&](int u, Unit& b) {
    const int uu = min(u, nu - 1);
#pragma unroll
    for (int t = 0; t < GU; ++t) b.w[t] = buf_ld16(w_rs, 16u * lane, (uint32_t)min(GU * uu + t, nkt - 1) * kTileBytes);
    const uint32_t at = (uint32_t)(uu / units_per_group) * N;
    b.s = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(s_rs, (int)(2u * s_col), (int)(2u * at), 0));
    if (ZERO) b.z = __builtin_amdgcn_raw_buffer_load_b32(z_rs, (int)s_col, (int)at, 0);
  };
  const u32x4_t flat = ZERO ? u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}
                            : u32x4_t{0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};
  f32x4_t acc[kChunks][4];
#pragma unroll
  for (int m = 0; m < kChunks; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](int u, const Unit& b) {
    float s[4], z[4];
    u32x4_t bw[GU][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = j & 1 ? bf16hi(b.s[j >> 1]) : bf16lo(b.s[j >> 1]);
      if (ZERO) z[j] = -16.0f - (float)((b.z >> (8 * j)) & 0xFFu);
#pragma unroll
      for (int t = 0; t < GU; ++t) bw[t][j] = int4_operand(b.w[t][j]);
    }
#pragma unroll
    for (int m = 0; m < kChunks; ++m) {
      if (m < nch) {
        u32x4_t a[GU];
#pragma unroll
        for (int t = 0; t < GU; ++t) a[t] = lds[u % kRing][t][m][lane];
        f32x4_t sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < GU; ++t) sum = mfma16x16x32(a[t], flat, sum);
        f32x4_t part[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) part[j][v] = ZERO ? z[j] * sum[v] : sum[v];
#pragma unroll
        for (int t = 0; t < GU; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[j] = mfma16x16x32(a[t], bw[t][j], part[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][j][v] = __builtin_fmaf(s[j], part[j][v], acc[m][j][v]);
          asm volatile("" : "+v"(acc[m][j]));
        }
      }
    }
  };

  Unit b0, b1;
  load_rows(0);
  if (nu > 1) load_rows(1);
  if (nu > 2) load_rows(2);
  load_weights(0, b0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  // Unit u: rows of u + 3 and weights of u + 1 are asked for; the rows of u + 1
  // (asked for in unit u - 2) have arrived when the unit ends.
  auto step = [&](int u, Unit& now, Unit& next) {
    if (u + 3 < nu) load_rows(u + 3);
    load_weights(u + 1, next);
    if (live) compute(u, now);
    // at most this unit's own loads may still be on their way
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(0) : "memory");
    __syncthreads();
  };
  int u = 0;
  for (; u + 2 <= nu; u += 2) {
    step(u, b0, b1);
    step(u + 1, b1, b0);
  }
  if (u < nu) step(u, b0, b1);
  if (!live || ncol >= N) return;   // no barrier follows

  float bb[4];
  {
    const uint32_t* bp = reinterpret_cast<const uint32_t*>(bias + (size_t)e * N + ncol);
    const uint32_t b01 = bp[0], b23 = bp[1];
    bb[0] = bf16lo(b01), bb[1] = bf16hi(b01), bb[2] = bf16lo(b23), bb[3] = bf16hi(b23);
  }
#pragma unroll
  for (int m = 0; m < kChunks; ++m)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int rr = m0 + 16 * m + 4 * g + v;
      if (rr < M) {
        const size_t orow = (size_t)(row0 + rr);
        const float o0 = acc[m][0][v] + bb[0], o1 = acc[m][1][v] + bb[1], o2 = acc[m][2][v] + bb[2],
                    o3 = acc[m][3][v] + bb[3];
        if (GATE_UP)
          *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(out) + orow * (N / 2) + ncol / 2) =
              pack_bf16x2(clamped_glu(o0, o1), clamped_glu(o2, o3));
        else
          *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + orow * N + ncol) = f32x4_t{o0, o1, o2, o3};
      }
    }
}

template <bool GATE_UP>
hipError_t launch(const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias, const int32_t* cnt,
                  const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k, int G, void* out,
                  hipStream_t stream) {
  const int64_t S = T * k;
  // 32-bit offsets into the token rows (of one expert, for down)
  if ((GATE_UP ? T : S) * K * 2 >= (int64_t)1 << 32) return hipErrorNotSupported;
  const int n_tiles = (N + kBN - 1) / kBN;
  const int64_t m_slots = (S + kBM - 1) / kBM + E;
  const int64_t grid = (n_tiles * m_slots + kXcds - 1) / kXcds * kXcds;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = G == 32 ? (Wz ? int4_gemm_kernel<GATE_UP, 1, true> : int4_gemm_kernel<GATE_UP, 1, false>)
                      : (Wz ? int4_gemm_kernel<GATE_UP, 2, true> : int4_gemm_kernel<GATE_UP, 2, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kGemmWaves * kWave), 0, stream, (const bf16_t*)A,
                     (const uint8_t*)Wq, (const uint16_t*)Ws, (const uint8_t*)Wz, (const bf16_t*)bias, cnt, off, rows, K,
                     N, E, k, T, n_tiles, G == 128 ? 2 : 1, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_int4_gate_up(const void* x, const void* Wq, const void* Ws, const void* Wz, const void* bgu,
                                    const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                                    int k, int I, int G, void* h, hipStream_t stream) {
  return launch<true>(x, Wq, Ws, Wz, bgu, cnt, off, rows, T, H, 2 * I, E, k, G, h, stream);
}

hipError_t launch_gemm_int4_down(const void* h, const void* Wq, const void* Ws, const void* Wz, const void* bd,
                                 const int32_t* cnt, const int32_t* off, int64_t T, int H, int E, int k, int I, int G,
                                 float* o, hipStream_t stream) {
  return launch<false>(h, Wq, Ws, Wz, bd, cnt, off, nullptr, T, I, H, E, k, G, o, stream);
}

}  // namespace moe
