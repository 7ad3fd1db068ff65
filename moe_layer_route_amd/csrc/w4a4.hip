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
// A workgroup owns one expert and 64 columns and walks K in stages of 512 values.
// Codes and scales go from HBM to LDS by direct loads, 256 bytes of a column an
// instruction row: reading 4 columns x 256 bytes at a time reaches 6.9 TB/s from
// registers alone, 16 columns x 64 bytes (the operand's own shape) 5.7, as columns
// of 1440 bytes begin anywhere in a cache line.  Wave w multiplies the w-th 128
// values of a stage.
//   Lane (g = lane / 16, c = lane % 16), column block j: column n0 + 4c + j, block
//   g of the wave's four.  So a lane's four accumulators are neighbouring columns
//   (gate and up of two pairs), their scales one word of the block-major scales,
//   and the 16 lanes of a row hold the 32 values of one block of h: its maximum is
//   four lane moves away, and h leaves as MXFP4 rows without a pass of its own.
//   In LDS a column (or row) has 256 bytes of a stage, its 16-byte chunk k at k ^ 4
//   (column / 4 % 4) (a row's at k ^ 4 (row % 4)): a wave's reads spread over all
//   banks.
// The partial sums of the waves are added in LDS in a fixed order.
//
// Bound by HBM: two stage buffers and three (16 or 32 rows a pass) or two workgroups
// a CU keep 66 to 78 KB of loads under way on it.  2880 x 5760, weights' bytes per
// second: 32 experts, 8 rows each 51 us, 5.6 TB/s (down 26 us); 128 experts, 8 rows
// 195 us, 5.8 TB/s (down 106).  With the operand's own shape, 16 columns x 64 bytes
// straight into registers, these took 69, 32, 262 and 132 us.  One token, four live
// experts: 9.7 and 8.3 us for 35 and 18 MB, each workgroup's chain of waits.
#include "few_slots.h"
#include "launch.h"
#include "mxfp4_device.h"

namespace moe {
namespace {

constexpr uint32_t kOutOfRange = 0x80000000u;   // any offset at or past this reads 0

#define LDS3 __attribute__((address_space(3)))

constexpr int kWaves = 4;
constexpr int kCols = 64;
constexpr int kStageBlocks = 16;                // blocks of 32 values a stage
constexpr int kColBytes = 16 * kStageBlocks;    // 256

// MG chunks of 16 rows a pass
template <int MG>
struct Shape {
  static constexpr int kRing = 2;               // stage buffers; the loads run a stage ahead
  static constexpr int kWBytes = kCols * kColBytes, kABytes = 16 * MG * kColBytes;
  static constexpr int kW = 0, kA = kW + kWBytes, kWs = kA + kABytes, kAs = kWs + kCols * kStageBlocks;
  static constexpr int kStage = kAs + 256 * kWaves;    // 22, 26 or 34 KB
  static constexpr int kLds = kRing * kStage;          // three, three or two workgroups a CU
  static constexpr int kLoads = 6 + MG;                // a wave and stage
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

// SLOTS: a workgroup column per token slot (M = 1, rows in slot order); gate_up picks
// the slot's expert from the logits, and one more column of workgroups writes the
// decision for the later launches, from which down reads it.
template <bool GATE_UP, int MG, bool SLOTS>
__global__ __launch_bounds__(kWaves * kWave) void w4a4_stream_kernel(
    const uint8_t* __restrict__ A,       // gate_up: x codes [T][K/2]; down: h codes [S][K/2] (permuted order)
    const uint8_t* __restrict__ As,      // [ceil(K/128)][a_rows][4]
    const uint8_t* __restrict__ Wq,      // [E][N][K/2]
    const uint8_t* __restrict__ Ws,      // [E][K/32][N]
    const bf16_t* __restrict__ bias,     // [E][N]
    const int32_t* __restrict__ cnt, const int32_t* __restrict__ off,
    const int32_t* __restrict__ rows,    // gate_up only: permuted slot ids
    int K, int N, int E, int kslots, int a_rows, int64_t S,
    void* __restrict__ out,              // gate_up: h codes [S][I/2]; down: float32 [S][N]
    uint8_t* __restrict__ out_s,         // gate_up: h scales [ceil(I/128)][S][4]
    Slots slots) {
  using C = Shape<MG>;
  __shared__ __align__(1024) char smem_g[C::kLds];
  LDS3 char* smem = (LDS3 char*)smem_g;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int e, M = 1, row0 = blockIdx.y;
  if constexpr (SLOTS && GATE_UP) {
    const int t = (int)blockIdx.y / kslots, j = (int)blockIdx.y % kslots;
    if ((int)blockIdx.x * kCols >= N) {                    // block-uniform
      if (j == 0 && wave == 0) write_decision(slots, t, E, lane);
      return;
    }
    e = slot_expert(slots, t, j, E, lane);
  } else if constexpr (SLOTS) {
    e = slots.ids[blockIdx.y];
  } else {
    e = S < E ? live_expert(cnt, E, blockIdx.y, lane) : (int)blockIdx.y;
    if (e < 0) return;                                     // block-uniform
    M = cnt[e];
    if (M == 0) return;                                    // block-uniform
    row0 = off[e];
  }
  const int nblk = K / 32;
  const int g = lane >> 4, c = lane & 15;
  const int n0 = blockIdx.x * kCols;
  const int ncol = n0 + 4 * c;
  // N % 32 == 0: a lane's four columns are all in range or all out of it
  const bool col_ok = ncol < N;
  const uint32_t row_bytes = (uint32_t)K / 2;
  const int ns = (nblk + kStageBlocks - 1) / kStageBlocks;

  // ---- direct-load assignments: wave w fills columns 16w .. 16w + 15, four an
  // instruction (column 16w + 4i + l / 16, chunk l % 16 ^ 4 i), the rows 4 MG w ..
  // likewise, its own blocks' weight scales (block l / 16, four columns a lane) and
  // its rows' scales (row l / 4, group l % 4 of the stage, the first 16 MG lanes).
  // What is past the edges is sent out of range and lands as 0. ----
  const u32x4_t w_rs = rsrc_words(Wq + (size_t)e * N * row_bytes, 0x7FFFFFFFu);
  const u32x4_t ws_rs = rsrc_words(Ws + (size_t)e * nblk * N, 0x7FFFFFFFu);
  const u32x4_t a_rs = rsrc_words(A, 0x7FFFFFFFu);
  const u32x4_t as_rs = rsrc_words(As, 0x7FFFFFFFu);
  uint32_t w_off[4];
  int w_chunk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 16 * wave + 4 * i + g;
    w_chunk[i] = c ^ (4 * i);
    w_off[i] = n < N ? (uint32_t)n * row_bytes + 16u * (uint32_t)w_chunk[i] : kOutOfRange;
  }
  const uint32_t s_col = (uint32_t)min(ncol, N - 4);
  const uint32_t ws_off = col_ok ? (uint32_t)g * (uint32_t)N + (uint32_t)ncol : kOutOfRange;
  const int a_chunk = c ^ (4 * g);

  for (int r0 = 0; r0 < M; r0 += 16 * MG) {
    const int nch = min(MG, (M - r0 + 15) / 16);           // block-uniform
    auto load_w = [&](int s, int buf) {
      const uint32_t at = lds0 + buf * C::kStage;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dma16(w_rs, kStageBlocks * s + w_chunk[i] < nblk ? w_off[i] : kOutOfRange, (uint32_t)(kColBytes * s),
              at + C::kW + (16 * wave + 4 * i) * kColBytes);
      const int b = kStageBlocks * s + 4 * wave;
      dma4(ws_rs, b + g < nblk ? ws_off : kOutOfRange, (uint32_t)b * (uint32_t)N, at + C::kWs + 256 * wave);
    };
    // the first stage's weights are asked for ahead of the rows
    load_w(0, 0);
    // The wave's rows, as scalars (vector loads would be counted with the direct
    // loads): 4 MG of them; rows past M feed outputs that are not stored.
    uint32_t a_off[MG], as_off = kOutOfRange;
#pragma unroll
    for (int q = 0; q < MG; ++q) {
      uint32_t row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = row0 + min(r0 + 4 * MG * wave + 4 * q + i, M - 1);
        row[i] = !GATE_UP ? (uint32_t)m
                 : SLOTS  ? (uint32_t)(m / kslots)
                          : (uint32_t)(((const __attribute__((address_space(4))) int32_t*)rows)[m] / kslots);
      }
      auto pick = [&](int i) {
        const uint32_t lo = i == 0 ? row[0] : row[1], hi = i == 2 ? row[2] : row[3];
        return i < 2 ? lo : hi;
      };
      a_off[q] = pick(g) * row_bytes + 16u * (uint32_t)a_chunk;
      if (lane >> 4 == q) as_off = ((uint32_t)(lane & 3) * (uint32_t)a_rows + pick((lane >> 2) & 3)) * 4u;
    }
    auto load_a = [&](int s, int buf) {
      const uint32_t at = lds0 + buf * C::kStage;
#pragma unroll
      for (int q = 0; q < MG; ++q)
        dma16(a_rs, kStageBlocks * s + a_chunk < nblk ? a_off[q] : kOutOfRange, (uint32_t)(kColBytes * s),
              at + C::kA + (4 * MG * wave + 4 * q) * kColBytes);
      dma4(as_rs, kStageBlocks * s + 4 * (lane & 3) < nblk ? as_off : kOutOfRange, (uint32_t)(4 * s) * (uint32_t)a_rows * 4u,
           at + C::kAs + 256 * wave);
    };
    load_a(0, 0);

    f32x4_t acc[MG][4];
#pragma unroll
    for (int q = 0; q < MG; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[q][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int s = 0; s < ns; ++s) {
      const int buf = s & 1;
      // stage s + 1 into the other buffer (its reads ended before the last barrier);
      // past the last stage the loads are out of range
      load_w(s + 1, buf ^ 1);
      load_a(s + 1, buf ^ 1);
      if constexpr (MG == 1) asm volatile("s_waitcnt vmcnt(7)" ::: "memory");
      else if constexpr (MG == 2) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(10)" ::: "memory");
      static_assert(C::kLoads == 6 + MG, "the waits count the loads of one stage");
      __builtin_amdgcn_s_barrier();
      const LDS3 char* at = smem + buf * C::kStage;
      const bool in = kStageBlocks * s + 4 * wave + g < nblk;   // no caller's byte past K is used: 255 would be a NaN
      u32x4_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = *(const LDS3 u32x4_t*)(at + C::kW + (4 * c + j) * kColBytes + 16 * ((4 * wave + g) ^ (4 * (c & 3))));
      const uint32_t sw = *(const LDS3 uint32_t*)(at + C::kWs + (4 * wave + g) * kCols + 4 * c);
#pragma unroll
      for (int q = 0; q < MG; ++q) {
        const int r = 16 * q + c;
        const u32x4_t a = *(const LDS3 u32x4_t*)(at + C::kA + r * kColBytes + 16 * ((4 * wave + g) ^ (4 * (r & 3))));
        uint32_t sa = *(const LDS3 uint8_t*)(at + C::kAs + 256 * (r / (4 * MG)) + 16 * (r % (4 * MG)) + 4 * wave + g);
        sa = in ? sa : 0u;
        acc[q][0] = mfma_fp4_16<0, 0>(a, w[0], acc[q][0], sa, sw);
        acc[q][1] = mfma_fp4_16<0, 1>(a, w[1], acc[q][1], sa, sw);
        acc[q][2] = mfma_fp4_16<0, 2>(a, w[2], acc[q][2], sa, sw);
        acc[q][3] = mfma_fp4_16<0, 3>(a, w[3], acc[q][3], sa, sw);
      }
      // every wave has read its part before the next stage's loads go there
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // the stage buffers now hold one chunk's partial sums a wave
    LDS3 float (*red)[4][4][kWave] = (LDS3 float (*)[4][4][kWave])smem;

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
                  const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k, int64_t near,
                  void* out, void* out_s, const Slots* slots, hipStream_t stream) {
  const int64_t S = T * k, a_rows = GATE_UP ? T : S;
  // 32-bit buffer offsets: the token codes and one expert's codes below 2 GiB,
  // so an offset at kOutOfRange never comes back into range
  if (a_rows * K / 2 >= ((int64_t)1 << 31) || (int64_t)N * K / 2 >= ((int64_t)1 << 31)) return hipErrorNotSupported;
  const int columns = (N + kCols - 1) / kCols;
  const dim3 grid((unsigned)(columns + (slots && GATE_UP ? 1 : 0)), (unsigned)(slots || S < E ? S : E));
  // Rows a pass by the mean rows an expert: 16, 32 or 64.  More rows cost LDS (two
  // instead of three workgroups a CU at 64) and reads of rows that are not there;
  // fewer cost another pass over the weights.  gate_up of 2880 x 5760, 16 / 32 / 64:
  // 32 experts, 8 rows each 51 / 54 / 66 us, 12: 58 / 54 / 64, 24: 92 / 63 / 69, 32:
  // 105 / 78 / 72; 128 experts, 8: 196 / 200 / 236, 16: 265 / 219 / 251, 32: 408 /
  // 301 / 278.
  auto kern = slots                  ? w4a4_stream_kernel<GATE_UP, 1, true>
              : near <= 10 * (int64_t)E ? w4a4_stream_kernel<GATE_UP, 1, false>
              : near <= 27 * (int64_t)E ? w4a4_stream_kernel<GATE_UP, 2, false>
                                     : w4a4_stream_kernel<GATE_UP, 4, false>;
  hipLaunchKernelGGL(kern, grid, dim3(kWaves * kWave), 0, stream, (const uint8_t*)A, (const uint8_t*)As,
                     (const uint8_t*)Wq, (const uint8_t*)Ws, (const bf16_t*)bias, cnt, off, rows, K, N, E, k,
                     (int)a_rows, S, out, (uint8_t*)out_s, slots ? *slots : Slots{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4a4_gate_up(const void* xq, const void* sx, const void* Wq, const void* Ws, const void* bgu,
                               const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                               int k, int I, int64_t near, void* hq, void* sh, hipStream_t stream) {
  return launch<true>(xq, sx, Wq, Ws, bgu, cnt, off, rows, T, H, 2 * I, E, k, near, hq, sh, nullptr, stream);
}

hipError_t launch_w4a4_down(const void* hq, const void* sh, const void* Wq, const void* Ws, const void* bd,
                            const int32_t* cnt, const int32_t* off, int64_t T, int H, int E, int k, int I,
                            int64_t near, float* o, hipStream_t stream) {
  return launch<false>(hq, sh, Wq, Ws, bd, cnt, off, nullptr, T, I, H, E, k, near, o, nullptr, nullptr, stream);
}

hipError_t launch_w4a4_slots(const void* x, const void* Wr, const void* br, const void* Wgu_q, const void* Wgu_s,
                             const void* bgu, const void* Wd_q, const void* Wd_s, const void* bd, int64_t T, int H, int E,
                             int k, int I, double* logits, int32_t* ids, float* w, int32_t* pos, void* xq, void* sx,
                             void* hq, void* sh, float* o, hipStream_t stream) {
  hipError_t e = launch_few_logits(x, Wr, br, T, H, E, logits, stream, xq, sx);
  if (e != hipSuccess) return e;
  const Slots slots{logits, ids, w, pos, k};
  e = launch<true>(xq, sx, Wgu_q, Wgu_s, bgu, nullptr, nullptr, nullptr, T, H, 2 * I, E, k, T * k, hq, sh, &slots, stream);
  if (e != hipSuccess) return e;
  return launch<false>(hq, sh, Wd_q, Wd_s, bd, nullptr, nullptr, nullptr, T, I, H, E, k, T * k, o, nullptr, &slots, stream);
}

}  // namespace moe
