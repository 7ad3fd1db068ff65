// W4A4 experts: products of MXFP4 rows and MXFP4 weights on the scaled matrix
// instructions, weights streamed (small token counts per expert).
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 5 (MXFP4 experts), section
// 2 (gate_up -> bias -> clamped GLU, down -> bias) and section 4 (block-uniform
// early exits, masked tails).
//
//   p[m][n] = sum over blocks b of 32 values: 2^(sa[m][b] + sw[b][n] - 254)
//             * sum_i a[m][32b + i] w[n][32b + i]
// The instruction takes the codes as they lie in memory and one scale byte a
// lane and operand, so nothing is converted: a step of 128 values of K is one
// 16-byte load for each 16 columns, one word that holds the four columns'
// scales, the token rows' codes and scale, and four matrix instructions per 16
// rows.
//
// A workgroup owns one expert and 64 columns; its four waves split K.  Lane
// (g = lane / 16, c = lane % 16), column block j: column n0 + 4c + j, block 4s +
// g of step s.  So a lane's four accumulators are neighbouring columns (gate and
// up of two pairs), their scales one word of the block-major scales, and the 16
// lanes of a row hold the 32 values of one block of h: its maximum is four lane
// moves away, and h leaves as MXFP4 rows without a pass of its own.
// The partial sums of the waves are added in LDS in a fixed order.
#include "launch.h"
#include "mxfp4_device.h"

namespace moe {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4_t buf_ld16(rsrc_t r, uint32_t voff) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, 0, 0));
}
constexpr uint32_t kOutOfRange = 0x80000000u;   // any offset at or past this reads 0

constexpr int kWaves = 4;
constexpr int kCols = 64;

// one step's loads: codes and scales of the lane's four columns, and of MG rows
template <int MG>
struct Step {
  u32x4_t w[4];
  uint32_t ws;
  u32x4_t a[MG];
  uint32_t as[MG];
};

// The y-th expert with rows (every lane of the wave gets it), -1 past the last.
__device__ __forceinline__ int live_expert(const int32_t* __restrict__ cnt, int E, int y, int lane) {
  int live[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    live[i] = e < E && cnt[e] > 0;
    sum += live[i];
  }
  int at = wave_incl_scan(sum, lane) - sum, found = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (live[i] && at == y) found = 4 * lane + i;
    at += live[i];
  }
  const uint64_t who = __ballot(found >= 0);
  if (who == 0) return -1;
  return __builtin_amdgcn_readfirstlane(__shfl(found, __ffsll((unsigned long long)who) - 1, kWave));
}

// MG: chunks of 16 rows a pass; D: steps in flight; WG: workgroups a CU.
template <bool GATE_UP, int MG, int D, int WG>
__global__ __launch_bounds__(kWaves * kWave, WG) void w4a4_stream_kernel(
    const uint8_t* __restrict__ A,       // gate_up: x codes [T][K/2]; down: h codes [S][K/2] (permuted order)
    const uint8_t* __restrict__ As,      // [ceil(K/128)][a_rows][4]
    const uint8_t* __restrict__ Wq,      // [E][N][K/2]
    const uint8_t* __restrict__ Ws,      // [E][K/32][N]
    const bf16_t* __restrict__ bias,     // [E][N]
    const int32_t* __restrict__ cnt, const int32_t* __restrict__ off,
    const int32_t* __restrict__ rows,    // gate_up only: permuted slot ids
    int K, int N, int E, int kslots, int a_rows, int64_t S,
    void* __restrict__ out,              // gate_up: h codes [S][I/2]; down: float32 [S][N]
    uint8_t* __restrict__ out_s) {       // gate_up: h scales [ceil(I/128)][S][4]
  __shared__ float red[kWaves][4][4][kWave];   // 16 KB: one chunk's partial sums per wave

  const int lane = threadIdx.x & (kWave - 1);
  const int e = S < E ? live_expert(cnt, E, blockIdx.y, lane) : (int)blockIdx.y;
  if (e < 0) return;                                       // block-uniform
  const int M = cnt[e];
  if (M == 0) return;                                      // block-uniform
  const int row0 = off[e];
  const int nblk = K / 32;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = lane >> 4, c = lane & 15;
  const int n0 = blockIdx.x * kCols;
  const int ncol = n0 + 4 * c;
  // N % 32 == 0: a lane's four columns are all in range or all out of it
  const bool col_ok = ncol < N;

  const uint32_t row_bytes = (uint32_t)K / 2;
  const rsrc_t w_rs = make_rsrc(Wq + (size_t)e * N * row_bytes, (uint32_t)N * row_bytes);
  const rsrc_t ws_rs = make_rsrc(Ws + (size_t)e * nblk * N, (uint32_t)(nblk * N));
  const rsrc_t a_rs = make_rsrc(A, (uint32_t)((size_t)a_rows * row_bytes));
  const int steps = (nblk + 3) / 4;
  const rsrc_t as_rs = make_rsrc(As, (uint32_t)((size_t)steps * a_rows * 4));
  const uint32_t s_col = (uint32_t)min(ncol, N - 4);
  uint32_t w_off[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w_off[j] = (uint32_t)min(ncol + j, N - 1) * row_bytes + 16u * g;
  const int begin = steps * wave / kWaves, end = steps * (wave + 1) / kWaves;

  for (int r0 = 0; r0 < M; r0 += 16 * MG) {
    const int nch = min(MG, (M - r0 + 15) / 16);           // block-uniform
    f32x4_t acc[MG][4];
#pragma unroll
    for (int q = 0; q < MG; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[q][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Blocks past K and steps past this wave's are sent out of range: codes and
    // scales 0 (no caller's padding byte, which may be a NaN, is read).
    auto load_w = [&](int s, Step<MG>& t) {
      const bool in = s < end && 4 * s + g < nblk;
#pragma unroll
      for (int j = 0; j < 4; ++j) t.w[j] = buf_ld16(w_rs, in ? w_off[j] + 64u * s : kOutOfRange);
      t.ws = __builtin_amdgcn_raw_buffer_load_b32(ws_rs, (int)(in ? (uint32_t)(4 * s + g) * N + s_col : kOutOfRange), 0, 0);
    };
    uint32_t a_row[MG];
// the first steps' weights are asked for ahead of the rows
    Step<MG> ring[D];
#pragma unroll
    for (int i = 0; i < D; ++i) load_w(begin + i, ring[i]);
#pragma unroll
    for (int q = 0; q < MG; ++q) {
      const int m = min(r0 + 16 * q + c, M - 1);           // rows past M feed outputs that are not stored
      a_row[q] = GATE_UP ? (uint32_t)(rows[row0 + m] / kslots) : (uint32_t)(row0 + m);
    }
    auto load_a = [&](int s, Step<MG>& t) {
      const bool in = s < end && 4 * s + g < nblk;
#pragma unroll
      for (int q = 0; q < MG; ++q) {
        t.a[q] = buf_ld16(a_rs, in ? a_row[q] * row_bytes + 64u * s + 16u * g : kOutOfRange);
        t.as[q] = __builtin_amdgcn_raw_buffer_load_b8(
            as_rs, (int)(in ? ((uint32_t)s * a_rows + a_row[q]) * 4u + g : kOutOfRange), 0, 0);
      }
    };
    auto multiply = [&](const Step<MG>& t) {
#pragma unroll
      for (int q = 0; q < MG; ++q) {
        if (q == 0 || q < nch) {
          acc[q][0] = mfma_fp4_16<0, 0>(t.a[q], t.w[0], acc[q][0], t.as[q], t.ws);
          acc[q][1] = mfma_fp4_16<0, 1>(t.a[q], t.w[1], acc[q][1], t.as[q], t.ws);
          acc[q][2] = mfma_fp4_16<0, 2>(t.a[q], t.w[2], acc[q][2], t.as[q], t.ws);
          acc[q][3] = mfma_fp4_16<0, 3>(t.a[q], t.w[3], acc[q][3], t.as[q], t.ws);
        }
      }
    };
#pragma unroll
    for (int i = 0; i < D; ++i) load_a(begin + i, ring[i]);
    for (int s = begin; s < end; s += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        multiply(ring[i]);
        load_w(s + i + D, ring[i]);
        load_a(s + i + D, ring[i]);
      }
    }

    float bb[4];
    {
      // two 4-byte reads: the bias is only guaranteed 4-byte alignment
      const uint32_t* bp = reinterpret_cast<const uint32_t*>(bias + (size_t)e * N + s_col);
      const uint32_t b01 = bp[0], b23 = bp[1];
      bb[0] = bf16lo(b01), bb[1] = bf16hi(b01), bb[2] = bf16lo(b23), bb[3] = bf16hi(b23);
    }
    // Sum of the four K parts (fixed order); wave w then finishes accumulator
    // element v = w (row 4g + w of each chunk) of all four column blocks.
#pragma unroll
    for (int q = 0; q < MG; ++q) {
      if (q < nch) {                                       // block-uniform
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) red[wave][j][v][lane] = acc[q][j][v];
        __syncthreads();
        float sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sum[j] = ((red[0][j][wave][lane] + red[1][j][wave][lane]) + red[2][j][wave][lane]) + red[3][j][wave][lane] + bb[j];
        const int m = r0 + 16 * q + 4 * g + wave;
        const size_t orow = (size_t)(row0 + m);
        if (GATE_UP) {
          // N % 64 == 0: every lane's columns are in range, and 16 lanes hold one block of h
          const uint32_t h = pack_bf16x2(clamped_glu(sum[0], sum[1]), clamped_glu(sum[2], sum[3]));
          const uint32_t s = mx_scale_byte(row16_max(abs_max2(h)));
          const uint32_t code = s == 255 ? 0u : encode2<0>(0u, h, ue8m0_to_f32(s)) & 0xFFu;
          if (m < M) {
            reinterpret_cast<uint8_t*>(out)[orow * (N / 4) + ncol / 4] = (uint8_t)code;
            const int b = n0 / 64;
            if (c == 0) out_s[((size_t)(b / 4) * S + orow) * 4 + b % 4] = (uint8_t)s;
          }
        } else if (m < M && col_ok) {
          *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + orow * N + ncol) =
              f32x4_t{sum[0], sum[1], sum[2], sum[3]};
        }
        __syncthreads();
      }
    }
  }
}

template <bool GATE_UP>
hipError_t launch(const void* A, const void* As, const void* Wq, const void* Ws, const void* bias, const int32_t* cnt,
                  const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k, void* out,
                  void* out_s, hipStream_t stream) {
  const int64_t S = T * k, a_rows = GATE_UP ? T : S;
  // 32-bit buffer offsets: the token codes and one expert's codes below 2 GiB,
  // so an offset at kOutOfRange never comes back into range
  if (a_rows * K / 2 >= ((int64_t)1 << 31) || (int64_t)N * K / 2 >= ((int64_t)1 << 31)) return hipErrorNotSupported;
  const dim3 grid((unsigned)((N + kCols - 1) / kCols), (unsigned)(S < E ? S : E));
  // Up to twelve rows an expert in the mean most fit one pass of 16; beyond, two
  // chunks a pass save the second reading of the weights (32 experts of 2880 x 5760:
  // T = 64 68.6 us against 74.1, T = 96 74.1 against 76.4, T = 128 96.8 against 78.8).
  auto kern = S <= 12 * (int64_t)E ? w4a4_stream_kernel<GATE_UP, 1, 3, 3> : w4a4_stream_kernel<GATE_UP, 2, 3, 2>;
  hipLaunchKernelGGL(kern, grid, dim3(kWaves * kWave), 0, stream, (const uint8_t*)A, (const uint8_t*)As,
                     (const uint8_t*)Wq, (const uint8_t*)Ws, (const bf16_t*)bias, cnt, off, rows, K, N, E, k,
                     (int)a_rows, S, out, (uint8_t*)out_s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4a4_gate_up(const void* xq, const void* sx, const void* Wq, const void* Ws, const void* bgu,
                               const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                               int k, int I, void* hq, void* sh, hipStream_t stream) {
  return launch<true>(xq, sx, Wq, Ws, bgu, cnt, off, rows, T, H, 2 * I, E, k, hq, sh, stream);
}

hipError_t launch_w4a4_down(const void* hq, const void* sh, const void* Wq, const void* Ws, const void* bd,
                            const int32_t* cnt, const int32_t* off, int64_t T, int H, int E, int k, int I, float* o,
                            hipStream_t stream) {
  return launch<false>(hq, sh, Wq, Ws, bd, cnt, off, nullptr, T, I, H, E, k, o, nullptr, stream);
}

}  // namespace moe
