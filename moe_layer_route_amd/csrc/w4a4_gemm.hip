// Tiled grouped GEMM of the W4A4 experts: MXFP4 rows times MXFP4 weights for
// larger token counts per expert (bound by the load path and the matrix cores).
//
// xserv "Phase 19: gpt-oss-20b MoE support": section 5 (MXFP4 experts, one
// batched launch), section 2 (gate_up -> bias -> GLU, down -> bias), section 4
// (early exits only when the whole workgroup leaves together; masked tails).
//
// Tile: 256 rows x 256 columns, K stages of 256 codes (one 128-byte line of
// every row and column), four waves in a 2 x 2 grid, each 128 x 128 = 4 x 4
// blocks of v_mfma_scale_f32_32x32x64_f8f6f4 (256 float32 accumulators a lane).
//   Staging: codes and scales HBM/L2 -> LDS by direct loads, two stage buffers
//   of 64 KB of codes and 4 KB of scales.  Row r's 16-byte chunk c (one block of
//   32 values) sits at slot c ^ ((r >> 1) & 7) of its 128 bytes.  LDS row 32q +
//   t of a wave's 128 columns is column 4t + q, so that accumulator blocks q = 0
//   .. 3 of a lane are four neighbouring columns: two (gate, up) pairs, one
//   16-byte store of down, and one word of the block-major weight scales.
//   Steps: step j of a stage has the blocks j (lanes 0-31) and 4 + j (lanes
//   32-63) of the stage's eight; the product only needs both operands to agree.
//   So a lane's four row scales of a stage are one word of the rows' scale
//   layout (its group of four blocks), step j takes byte j of it, and column
//   block q takes byte q of the weight scales' word of block 4 (l / 32) + j:
//   8 scale words a lane and stage, picked by the instruction itself.
//   Stage s: after the barrier that ends stage s - 1, the loads of stage s + 1 go
//   into the other buffer; each wave waits for its own at the end of the stage
//   and the barrier makes all of them visible.
// Epilogue of gate_up: 16 lanes hold one block of h for a row: maximum by lane
// moves, codes by the conversion instruction, then a 4 x 4 byte transpose in each
// quad of lanes makes a lane's four bytes those of one row.
#include "launch.h"
#include "mxfp4_device.h"

namespace moe {
namespace {

#define LDS3 __attribute__((address_space(3)))

constexpr int kThreads = 256;
constexpr int kTile = 256;
constexpr int kStage = 256;                    // codes per K stage
constexpr int kRowBytes = kStage / 2;          // 128
constexpr int kOpBytes = kTile * kRowBytes;    // 32 KB: one operand of one stage
constexpr int kA = 0;                          // A of buffer b at b * 32 KB
constexpr int kB = 2 * kOpBytes;
constexpr int kAs = 4 * kOpBytes;              // row scales of buffer b: 2 groups x 256 rows x 4 bytes
constexpr int kAsBytes = 2 * kTile * 4;
constexpr int kBs = kAs + 2 * kAsBytes;        // weight scales of buffer b: 8 blocks x 256 columns
constexpr int kBsBytes = 8 * kTile;
constexpr int kLds = kBs + 2 * kBsBytes;       // 136 KB
constexpr int kMBlock = 1024;                  // M tiles per block of the tile order: all of an expert's
constexpr int kXcds = 8;
constexpr uint32_t kOOR = 0x80000000u;         // beyond every descriptor's range

template <bool GATE_UP>
__global__ __launch_bounds__(kThreads, 1) void w4a4_gemm_kernel(
    const uint8_t* __restrict__ A,       // gate_up: x codes [T][K/2]; down: h codes [S][K/2] (permuted order)
    const uint8_t* __restrict__ As,      // [ceil(K/128)][a_rows][4]
    const uint8_t* __restrict__ Wq,      // [E][N][K/2]
    const uint8_t* __restrict__ Ws,      // [E][K/32][N]
    const bf16_t* __restrict__ bias,     // [E][N] (interleaved gate/up for gate_up)
    const int32_t* __restrict__ cnt, const int32_t* __restrict__ off,
    const int32_t* __restrict__ rows,    // gate_up: permuted slot ids
    int K, int N, int E, int kslots, int a_rows, int64_t S, int n_tiles,
    void* __restrict__ out,              // gate_up: h codes [S][I/2]; down: float32 [S][N]
    uint8_t* __restrict__ out_s) {       // gate_up: h scales [ceil(I/128)][S][4]
  __shared__ __align__(1024) char smem_g[kLds];
  LDS3 char* smem = (LDS3 char*)smem_g;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave >> 1, wn = wave & 1;

  int e, m0, nt;
  if (!grouped_gemm_tile(cnt, E, kTile, n_tiles, kMBlock, lane, e, m0, nt)) return;   // workgroup-uniform
  const int n0 = nt * kTile;
  const int M = cnt[e];
  const int row0 = off[e];
  const int Kb = K / 2;
  const int nblk = K / 32;
  const int ns = (nblk + 7) / 8;

  // ---- direct-load assignments: wave w fills rows 64w .. 64w + 63 of both
  // tiles, eight rows an instruction; lane l takes row 8i + l / 8 of its
  // instruction i and chunk c = (l % 8) ^ ((r >> 1) & 7) of it.  What is past the
  // edges is sent out of range and lands as 0. ----
  const u32x4_t a_rs = rsrc_words(A, 0x7FFFFFFFu);
  const u32x4_t b_rs = rsrc_words(Wq + (size_t)e * N * Kb, 0x7FFFFFFFu);
  const u32x4_t as_rs = rsrc_words(As, 0x7FFFFFFFu);
  const u32x4_t bs_rs = rsrc_words(Ws + (size_t)e * nblk * N, 0x7FFFFFFFu);
  const int lc[2] = {(lane & 7) ^ ((lane >> 4) & 7), (lane & 7) ^ (((lane >> 4) + 4) & 7)};  // even, odd i
  uint32_t a_off[8], b_off[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 64 * wave + 8 * i + (lane >> 3);
    const uint32_t c16 = 16u * (uint32_t)lc[i & 1];
    const int m = m0 + r;
    if (m < M) {
      const uint32_t row = GATE_UP ? (uint32_t)(rows[row0 + m] / kslots) : (uint32_t)(row0 + m);
      a_off[i] = row * (uint32_t)Kb + c16;
    } else {
      a_off[i] = kOOR;
    }
    const int n = n0 + (r & ~127) + 4 * (r & 31) + ((r >> 5) & 3);
    b_off[i] = n < N ? (uint32_t)n * (uint32_t)Kb + c16 : kOOR;
  }
  // row scales: wave w, group h of the stage: rows 64w + lane
  uint32_t as_off = kOOR;
  {
    const int m = m0 + 64 * wave + lane;
    if (m < M) as_off = 4u * (GATE_UP ? (uint32_t)(rows[row0 + m] / kslots) : (uint32_t)(row0 + m));
  }
  // weight scales: waves 0 and 1, four blocks each: block 4w + l / 16, 16 columns
  const int bs_col = n0 + 16 * (lane & 15);
  const uint32_t bs_off = bs_col < N ? (uint32_t)(4 * (wave & 1) + (lane >> 4)) * (uint32_t)N + (uint32_t)bs_col : kOOR;

  auto dma = [&](int st, int buf, int i, bool b_side) {
    const int k0 = st * kRowBytes;
    const uint32_t base = b_side ? b_off[i] : a_off[i];
    const uint32_t voff = k0 + 16 * lc[i & 1] < Kb ? base : kOOR;
    const uint32_t lds = lds0 + (b_side ? kB : kA) + buf * kOpBytes + (64 * wave + 8 * i) * kRowBytes;
    dma16(b_side ? b_rs : a_rs, voff, (uint32_t)k0, lds);
  };
  auto dma_scales = [&](int st, int buf) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int group = 2 * st + h;
      dma4(as_rs, 4 * group < nblk ? as_off : kOOR, (uint32_t)group * (uint32_t)a_rows * 4u,
           lds0 + kAs + buf * kAsBytes + h * kTile * 4 + 64 * wave * 4);
    }
    if (wave < 2)   // wave-uniform
      dma16(bs_rs, 8 * st + 4 * wave + (lane >> 4) < nblk ? bs_off : kOOR, (uint32_t)(8 * st) * (uint32_t)N,
            lds0 + kBs + buf * kBsBytes + wave * 4 * kTile);
  };

  // ---- fragment reads: step j has chunk j (lanes 0-31) or 4 + j (lanes 32-63) ----
  const int fr = lane & 31, fg = lane >> 5;
  uint32_t a_rd[4], b_rd[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t xo = 16u * (uint32_t)((4 * fg + j) ^ ((fr >> 1) & 7));
    a_rd[j] = (uint32_t)(kA + (128 * wm + fr) * kRowBytes) + xo;
    b_rd[j] = (uint32_t)(kB + (128 * wn + fr) * kRowBytes) + xo;
  }
  auto read_frag = [&](int buf, int j, int q, bool b_side) -> u32x4_t {
    return *(const LDS3 u32x4_t*)(smem + (b_side ? b_rd[j] : a_rd[j]) + buf * kOpBytes + q * 32 * kRowBytes);
  };
  const uint32_t as_rd = (uint32_t)(kAs + fg * kTile * 4 + (128 * wm + fr) * 4);
  const uint32_t bs_rd = (uint32_t)(kBs + 4 * fg * kTile + 128 * wn + 4 * fr);

  f32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // a stage's scale words: row block i (byte: step), step j (byte: column block)
  struct Scales {
    uint32_t a[4], b[4];
  };
  Scales sc = {}, last;
  auto read_scales = [&](int s, int buf) {
    // no byte past K is used: it is a caller's, and 255 would be a NaN
    const int live = nblk - 8 * s - 4 * fg;
    const uint32_t mask = live >= 4 ? 0xFFFFFFFFu : live <= 0 ? 0u : (1u << (8 * live)) - 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sc.a[i] = *(const LDS3 uint32_t*)(smem + as_rd + buf * kAsBytes + i * 32 * 4) & mask;
      sc.b[i] = *(const LDS3 uint32_t*)(smem + bs_rd + buf * kBsBytes + i * kTile);
    }
  };
  // fragments in the order they are read (a0 b0 a1 b1 ...), each product as soon
  // as both its operands are there: slot u of four
#define MX_MFMA(J, I, Q) acc[I][Q] = mfma_fp4_32<J, Q>(fa[I], fb[Q], acc[I][Q], s4.a[I], s4.b[J])
#define MX_SLOT(J)                                                            \
  if (u == 0) {                                                               \
    MX_MFMA(J, 0, 0); MX_MFMA(J, 0, 1); MX_MFMA(J, 1, 0); MX_MFMA(J, 1, 1);   \
  } else if (u == 1) {                                                        \
    MX_MFMA(J, 0, 2); MX_MFMA(J, 1, 2); MX_MFMA(J, 2, 0); MX_MFMA(J, 2, 1);   \
  } else if (u == 2) {                                                        \
    MX_MFMA(J, 2, 2); MX_MFMA(J, 0, 3); MX_MFMA(J, 1, 3); MX_MFMA(J, 2, 3);   \
  } else {                                                                    \
    MX_MFMA(J, 3, 0); MX_MFMA(J, 3, 1); MX_MFMA(J, 3, 2); MX_MFMA(J, 3, 3);   \
  }
  auto slot = [&](int j, int u, const u32x4_t (&fa)[4], const u32x4_t (&fb)[4], const Scales& s4) {
    if (j == 0) {
      MX_SLOT(0)
    } else if (j == 1) {
      MX_SLOT(1)
    } else if (j == 2) {
      MX_SLOT(2)
    } else {
      MX_SLOT(3)
    }
  };

  // prologue: stage 0 into buffer 0
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    dma(0, 0, i, false);
    dma(0, 0, i, true);
  }
  dma_scales(0, 0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();

  u32x4_t fa0[4], fb0[4], fa1[4], fb1[4];
  // Step j of stage s in four slots: slot u reads fragments u of both operands
  // for step j and issues four products of the step before; the slots of the
  // first two steps also issue the loads of stage s + 1 (past the last: none).
  auto step = [&](int s, int buf, int j, u32x4_t (&fa_rd)[4], u32x4_t (&fb_rd)[4], const u32x4_t (&fa_mm)[4],
                  const u32x4_t (&fb_mm)[4], const Scales& s4, bool do_mfma) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (j < 2) {
        dma(s + 1, buf ^ 1, 4 * j + u, false);
        dma(s + 1, buf ^ 1, 4 * j + u, true);
        if (j == 1 && u == 3) dma_scales(s + 1, buf ^ 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      fa_rd[u] = read_frag(buf, j, u, false);
      fb_rd[u] = read_frag(buf, j, u, true);
      if (do_mfma) slot((j + 3) & 3, u, fa_mm, fb_mm, s4);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int s = 0; s < ns; ++s) {
    const int buf = s & 1;
    last = sc;
    read_scales(s, buf);
    step(s, buf, 0, fa0, fb0, fa1, fb1, last, s > 0);
    step(s, buf, 1, fa1, fb1, fa0, fb0, sc, true);
    step(s, buf, 2, fa0, fb0, fa1, fb1, sc, true);
    step(s, buf, 3, fa1, fb1, fa0, fb0, sc, true);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) slot(3, u, fa1, fb1, sc);

  // ---- epilogue.  Lane l, element v of block (i, q): row 32i + 8 (v / 4) + 4 (l
  // / 32) + v % 4, column 4 (l % 32) + q of the wave's 128. ----
  const int ncol = n0 + 128 * wn + 4 * fr;
  float bb[4];
  {
    const uint32_t* bp = reinterpret_cast<const uint32_t*>(bias + (size_t)e * N + min(ncol, N - 4));
    const uint32_t b01 = bp[0], b23 = bp[1];
    bb[0] = bf16lo(b01), bb[1] = bf16hi(b01), bb[2] = bf16lo(b23), bb[3] = bf16hi(b23);
  }
  if (GATE_UP) {
    const int b = (n0 + 128 * wn) / 64 + (fr >> 4);          // this lane's block of h
    const int l4 = lane & 3;
    const uint32_t pick = 0x01010101u * (uint32_t)l4 + 0x04000400u;   // bytes l4 of two words, twice
    uint8_t* codes = reinterpret_cast<uint8_t*>(out);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v4 = 0; v4 < 4; ++v4) {
        const int m4 = m0 + 128 * wm + 32 * i + 8 * v4 + 4 * fg;     // rows m4 .. m4 + 3
        uint32_t c4 = 0, s4 = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int v = 4 * v4 + r;
          const uint32_t h = pack_bf16x2(clamped_glu(acc[i][0][v] + bb[0], acc[i][1][v] + bb[1]),
                                         clamped_glu(acc[i][2][v] + bb[2], acc[i][3][v] + bb[3]));
          const uint32_t s = mx_scale_byte(row16_max(abs_max2(h)));
          const uint32_t c = s == 255 ? 0u : encode2<0>(0u, h, ue8m0_to_f32(s)) & 0xFFu;
          c4 |= c << (8 * r);
          s4 |= s << (8 * r);
        }
        // lane l4 of a quad: byte l4 (row m4 + l4) of the quad's four words
        const uint32_t q0 = moved<0x00>(c4), q1 = moved<0x55>(c4), q2 = moved<0xAA>(c4), q3 = moved<0xFF>(c4);
        const uint32_t lo = perm_b32(q1, q0, pick), hi = perm_b32(q3, q2, pick);
        const uint32_t word = pack_lo(lo, hi);
        const int m = m4 + l4;
        if (m < M && ncol < N) {
          const size_t orow = (size_t)(row0 + m);
          *reinterpret_cast<uint32_t*>(codes + orow * (N / 4) + (ncol & ~15) / 4) = word;
          if ((lane & 15) < 4) out_s[((size_t)(b / 4) * S + orow) * 4 + b % 4] = (uint8_t)(s4 >> (8 * l4));
        }
      }
  } else {
    if (ncol >= N) return;                                   // N % 32 == 0: four columns are all in or all out
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + 128 * wm + 32 * i + 8 * (v >> 2) + 4 * fg + (v & 3);
        if (m < M)
          *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + (size_t)(row0 + m) * N + ncol) =
              f32x4_t{acc[i][0][v] + bb[0], acc[i][1][v] + bb[1], acc[i][2][v] + bb[2], acc[i][3][v] + bb[3]};
      }
  }
}

template <bool GATE_UP>
hipError_t launch(const void* A, const void* As, const void* Wq, const void* Ws, const void* bias, const int32_t* cnt,
                  const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k, void* out, void* out_s,
                  hipStream_t stream) {
  const int64_t S = T * k, a_rows = GATE_UP ? T : S;
  // 32-bit buffer offsets: the token codes and one expert's codes below 2 GiB
  if (a_rows * K / 2 >= ((int64_t)1 << 31) || (int64_t)N * K / 2 >= ((int64_t)1 << 31)) return hipErrorNotSupported;
  const int n_tiles = (N + kTile - 1) / kTile;
  // at most sum_e ceil(cnt_e / 256) <= S / 256 + min(E, S) M tiles
  const int64_t tiles = (S / kTile + (S < E ? S : E)) * n_tiles;
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((w4a4_gemm_kernel<GATE_UP>), dim3((unsigned)grid), dim3(kThreads), 0, stream, (const uint8_t*)A,
                     (const uint8_t*)As, (const uint8_t*)Wq, (const uint8_t*)Ws, (const bf16_t*)bias, cnt, off, rows, K,
                     N, E, k, (int)a_rows, S, n_tiles, out, (uint8_t*)out_s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w4a4_gate_up(const void* xq, const void* sx, const void* Wq, const void* Ws, const void* bgu,
                                    const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                                    int k, int I, void* hq, void* sh, hipStream_t stream) {
  return launch<true>(xq, sx, Wq, Ws, bgu, cnt, off, rows, T, H, 2 * I, E, k, hq, sh, stream);
}

hipError_t launch_gemm_w4a4_down(const void* hq, const void* sh, const void* Wq, const void* Ws, const void* bd,
                                 const int32_t* cnt, const int32_t* off, int64_t T, int H, int E, int k, int I, float* o,
                                 hipStream_t stream) {
  return launch<false>(hq, sh, Wq, Ws, bd, cnt, off, nullptr, T, I, H, E, k, o, nullptr, stream);
}

}  // namespace moe
