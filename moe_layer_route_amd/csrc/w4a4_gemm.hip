// Tiled grouped GEMM of the W4A4 experts: MXFP4 rows times MXFP4 weights for
// larger token counts per expert (bound by the load path and the matrix cores).
//
// xserv "Phase 19: gpt-oss-20b MoE support": section 5 (MXFP4 experts, one
// batched launch), section 2 (gate_up -> bias -> GLU, down -> bias), section 4
// (early exits only when the whole workgroup leaves together; masked tails).
//
// Tile: 128 rows x 256 columns, K stages of 128 codes (64 bytes of every row and
// column), four waves in a 2 x 2 grid, each 64 x 128 = 2 x 4 blocks of
// v_mfma_scale_f32_32x32x64_f8f6f4 (128 float32 accumulators a lane).  A second
// kernel below has tiles of 256 x 256 and of 128 x 128; the launch says which is taken.
//   Staging: codes and scales HBM/L2 -> LDS by direct loads into a ring of three
//   stage buffers (24 KB of codes, 2 KB of scales each), two stages ahead; 78 KB, so
//   two workgroups share a CU and one multiplies while the other starts or ends.
//   Row r's 16-byte chunk c (one block of 32 values) sits at slot c ^ ((r >> 2) & 3)
//   of its 64 bytes.  LDS row 32q + t of a wave's 128 columns is column 4t + q, so
//   that accumulator blocks q = 0 .. 3 of a lane are four neighbouring columns: two
//   (gate, up) pairs, one 16-byte store of down, and one word of the block-major
//   weight scales.
//   Steps: step j of a stage has the blocks j (lanes 0-31) and 2 + j (lanes 32-63)
//   of the stage's four; the product only needs both operands to agree.  A lane's
//   row scales of a stage are one word of the rows' layout, shifted once by its
//   half, step j takes byte j of it, and column block q takes byte q of the weight
//   scales' word of block 2 (l / 32) + j: picked by the instruction itself.
//   Stage s: its loads were issued during stage s - 2; each wave waits for its own
//   at the end of stage s - 1 and the barrier makes all of them visible.
// What bounds them: the load path and the products in turn.  2880 x 5760, 512 rows an
// expert, 32 experts: 255 to 265 us, 2.1 PFLOP/s with either large tile, matrix pipes 26%
// busy at 2.1 GHz (down 166 and 149 us, 1.6 and 1.8 PFLOP/s).  One expert of 16384 rows
// by these tiles: 222 us, without the loads 143, without the products 176, without both
// 89.  With stages of this size, tiles of 256 x 256 by eight waves took 293 us where
// these took 256; with whole lines and four waves, one a SIMD, 316.
#include "launch.h"
#include "mxfp4_device.h"

#include <type_traits>

namespace moe {
namespace {

#define LDS3 __attribute__((address_space(3)))

constexpr int kThreads = 256;
constexpr int kBM = 128, kBN = 256;
constexpr int kStage = 128;                    // codes per K stage: one word of row scales
constexpr int kRowBytes = kStage / 2;          // 64
constexpr int kRing = 3;                       // stage buffers; the loads run kRing - 1 stages ahead
constexpr int kABytes = kBM * kRowBytes;       // 8 KB
constexpr int kBBytes = kBN * kRowBytes;       // 16 KB
constexpr int kA = 0;                          // A of buffer b at b * 8 KB
constexpr int kB = kRing * kABytes;
constexpr int kAs = kB + kRing * kBBytes;      // row scales of buffer b: 32 words for each wave, 256 bytes apart
constexpr int kAsBytes = 1024;
constexpr int kBs = kAs + kRing * kAsBytes;    // weight scales of buffer b: 4 blocks x 256 columns
constexpr int kBsBytes = 4 * kBN;
constexpr int kLds = kBs + kRing * kBsBytes;   // 78 KB: two workgroups a CU
constexpr int kMBlock = 1024;                  // M tiles per block of the tile order: all of an expert's
constexpr int kXcds = 8;
constexpr uint32_t kOOR = 0x80000000u;         // beyond every descriptor's range

// Four rows m4 .. m4 + 3 of h from a lane's four neighbouring columns (two gate, up
// pairs) of each, p[column][row] without the bias.  16 lanes hold one block of h for
// a row: maximum by lane moves, codes by the conversion instruction, then a 4 x 4
// byte transpose in each quad of lanes makes a lane's four bytes those of one row.
__device__ __forceinline__ void store_glu_quad(const f32x4_t (&p)[4], const float (&bb)[4], int m4, int M, int row0,
                                               int ncol, int N, int lane, uint8_t* __restrict__ codes,
                                               uint8_t* __restrict__ out_s, int64_t S) {
  const int b = ncol / 64;                                 // this lane's block of h
  const int l4 = lane & 3;
  const uint32_t pick = 0x01010101u * (uint32_t)l4 + 0x04000400u;   // bytes l4 of two words, twice
  uint32_t c4 = 0, s4 = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t h = pack_bf16x2(clamped_glu(p[0][r] + bb[0], p[1][r] + bb[1]),
                                   clamped_glu(p[2][r] + bb[2], p[3][r] + bb[3]));
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

template <bool GATE_UP>
__global__ __launch_bounds__(kThreads, 2) void w4a4_gemm_kernel(
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
  if (!grouped_gemm_tile(cnt, E, kBM, n_tiles, kMBlock, lane, e, m0, nt)) return;   // workgroup-uniform
  const int n0 = nt * kBN;
  const int M = cnt[e];
  const int row0 = off[e];
  const int Kb = K / 2;
  const int nblk = K / 32;
  const int ns = (nblk + 3) / 4;

  // ---- direct-load assignments: wave w fills rows 32w .. 32w + 31 of A and 64w
  // .. 64w + 63 of B, sixteen rows an instruction; lane l takes row 16i + l / 4 of
  // its instruction i and chunk c = (l % 4) ^ ((r >> 2) & 3) of it.  What is past
  // the edges is sent out of range and lands as 0. ----
  const u32x4_t a_rs = rsrc_words(A, 0x7FFFFFFFu);
  const u32x4_t b_rs = rsrc_words(Wq + (size_t)e * N * Kb, 0x7FFFFFFFu);
  const u32x4_t as_rs = rsrc_words(As, 0x7FFFFFFFu);
  const u32x4_t bs_rs = rsrc_words(Ws + (size_t)e * nblk * N, 0x7FFFFFFFu);
  const int lc = (lane & 3) ^ ((lane >> 4) & 3);
  uint32_t a_off[2], b_off[4];
  auto row_of = [&](int m) {
    return GATE_UP ? (uint32_t)(rows[row0 + m] / kslots) : (uint32_t)(row0 + m);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = m0 + 32 * wave + 16 * i + (lane >> 2);
    a_off[i] = m < M ? row_of(m) * (uint32_t)Kb + 16u * lc : kOOR;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 64 * wave + 16 * i + (lane >> 2);
    const int n = n0 + (r & ~127) + 4 * (r & 31) + ((r >> 5) & 3);
    b_off[i] = n < N ? (uint32_t)n * (uint32_t)Kb + 16u * lc : kOOR;
  }
  // row scales: rows 32w + lane of the first 32 lanes (the others fill the gap
  // behind them); weight scales: block w of the stage, four columns a lane
  uint32_t as_off = kOOR;
  {
    const int m = m0 + 32 * wave + lane;
    if (lane < 32 && m < M) as_off = 4u * row_of(m);
  }
  const uint32_t bs_off = n0 + 4 * lane < N ? (uint32_t)wave * (uint32_t)N + (uint32_t)(n0 + 4 * lane) : kOOR;

  // eight loads a wave and stage (the waits below count them)
  auto dma = [&](int st, int buf, int i) {   // 0, 1: A; 2 .. 5: B; 6, 7: scales
    const int k0 = st * kRowBytes;
    if (i < 2)
      dma16(a_rs, k0 + 16 * lc < Kb ? a_off[i] : kOOR, (uint32_t)k0,
            lds0 + kA + buf * kABytes + (32 * wave + 16 * i) * kRowBytes);
    else if (i < 6)
      dma16(b_rs, k0 + 16 * lc < Kb ? b_off[i - 2] : kOOR, (uint32_t)k0,
            lds0 + kB + buf * kBBytes + (64 * wave + 16 * (i - 2)) * kRowBytes);
    else if (i == 6)
      dma4(as_rs, 4 * st < nblk ? as_off : kOOR, (uint32_t)st * (uint32_t)a_rows * 4u,
           lds0 + kAs + buf * kAsBytes + 256 * wave);
    else
      dma4(bs_rs, 4 * st + wave < nblk ? bs_off : kOOR, (uint32_t)(4 * st) * (uint32_t)N,
           lds0 + kBs + buf * kBsBytes + wave * kBN);
  };

  // ---- fragment reads: step j has chunk j (lanes 0-31) or 2 + j (lanes 32-63) ----
  const int fr = lane & 31, fg = lane >> 5;
  uint32_t a_rd[2], b_rd[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t xo = 16u * (uint32_t)((2 * fg + j) ^ ((fr >> 2) & 3));
    a_rd[j] = (uint32_t)(kA + (64 * wm + fr) * kRowBytes) + xo;
    b_rd[j] = (uint32_t)(kB + (128 * wn + fr) * kRowBytes) + xo;
  }
  auto read_a = [&](int buf, int j, int i) -> u32x4_t {
    return *(const LDS3 u32x4_t*)(smem + a_rd[j] + buf * kABytes + i * 32 * kRowBytes);
  };
  auto read_b = [&](int buf, int j, int q) -> u32x4_t {
    return *(const LDS3 u32x4_t*)(smem + b_rd[j] + buf * kBBytes + q * 32 * kRowBytes);
  };
  const uint32_t as_rd = (uint32_t)(kAs + 512 * wm + fr * 4);
  const uint32_t bs_rd = (uint32_t)(kBs + 2 * fg * kBN + 128 * wn + 4 * fr);

  f32x16_t acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // a stage's scale words: row block i (byte: step), step j (byte: column block)
  struct Scales {
    uint32_t a[2], b[2];
  };
  Scales sc = {}, last;
  auto read_scales = [&](int s, int buf) {
    // no byte past K is used: it is a caller's, and 255 would be a NaN
    const int live = nblk - 4 * s;
    const uint32_t mask = live >= 4 ? 0xFFFFFFFFu : (1u << (8 * live)) - 1u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sc.a[i] = (*(const LDS3 uint32_t*)(smem + as_rd + buf * kAsBytes + i * 256) & mask) >> (16 * fg);
      sc.b[i] = *(const LDS3 uint32_t*)(smem + bs_rd + buf * kBsBytes + i * kBN);
    }
  };
  // fragments in the order they are read (a0 b0 a1 b1 b2 b3), two products behind
  // each, in three slots
#define MX_MFMA(J, I, Q) \
  if constexpr (I < NI) acc[I][Q] = mfma_fp4_32<J, Q>(fa[I], fb[Q], acc[I][Q], s4.a[I], s4.b[J])
#define MX_SLOT(J)                                          \
  if (u == 0) {                                             \
    MX_MFMA(J, 0, 0);                                       \
    MX_MFMA(J, 1, 0);                                       \
  } else if (u == 1) {                                      \
    MX_MFMA(J, 0, 1); MX_MFMA(J, 1, 1); MX_MFMA(J, 0, 2);   \
  } else {                                                  \
    MX_MFMA(J, 1, 2); MX_MFMA(J, 0, 3); MX_MFMA(J, 1, 3);   \
  }
  // prologue: stages 0 .. kRing - 2
#pragma unroll
  for (int st = 0; st < kRing - 1; ++st)
#pragma unroll
    for (int i = 0; i < 8; ++i) dma(st, st, i);
  asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
  __builtin_amdgcn_s_barrier();

  // The loop for the NI row blocks of 32 that the wave has rows in: the products of the
  // others are left out.
  auto loop = [&](auto ni_c) {
    constexpr int NI = decltype(ni_c)::value;
    auto slot = [&](int j, int u, const u32x4_t (&fa)[2], const u32x4_t (&fb)[4], const Scales& s4) {
      if (j == 0) {
        MX_SLOT(0)
      } else {
        MX_SLOT(1)
      }
    };

    u32x4_t fa0[2], fb0[4], fa1[2], fb1[4];
    // Step j of stage s in three slots: slot u reads two fragments for step j,
    // issues loads of stage s + kRing - 1 into the buffer that stage s - 1 left at
    // the last barrier, and products of the step before.
    auto step = [&](int s, int buf, int nbuf, int j, u32x4_t (&fa_rd)[2], u32x4_t (&fb_rd)[4], const u32x4_t (&fa_mm)[2],
                    const u32x4_t (&fb_mm)[4], const Scales& s4, bool do_mfma) {
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        if (s + kRing - 1 < ns) {
          dma(s + kRing - 1, nbuf, 4 * j + u);
          if (u == 2) dma(s + kRing - 1, nbuf, 4 * j + 3);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (NI == 0) {
        } else if (u == 0) {
          fa_rd[0] = read_a(buf, j, 0);
          fb_rd[0] = read_b(buf, j, 0);
        } else if (u == 1) {
          if (NI > 1) fa_rd[1] = read_a(buf, j, 1);
          fb_rd[1] = read_b(buf, j, 1);
        } else {
          fb_rd[2] = read_b(buf, j, 2);
          fb_rd[3] = read_b(buf, j, 3);
        }
        if (do_mfma) slot(j ^ 1, u, fa_mm, fb_mm, s4);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int buf = 0, nbuf = kRing - 1;
    for (int s = 0; s < ns; ++s) {
      last = sc;
      if (NI > 0) read_scales(s, buf);
      step(s, buf, nbuf, 0, fa0, fb0, fa1, fb1, last, s > 0);
      step(s, buf, nbuf, 1, fa1, fb1, fa0, fb0, sc, true);
      // stage s + 1 has landed when only the loads of the stage behind it, if any, are out
      if (s + kRing - 1 < ns) asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      nbuf = buf;
      buf = buf == kRing - 1 ? 0 : buf + 1;
    }
#pragma unroll
    for (int u = 0; u < 3; ++u) slot(1, u, fa1, fb1, sc);
  };
  const int ni = min(2, max(0, (M - m0 - 64 * wm + 31) / 32));   // wave-uniform
  if (ni == 2) loop(std::integral_constant<int, 2>{});
  else if (ni == 1) loop(std::integral_constant<int, 1>{});
  else loop(std::integral_constant<int, 0>{});
  // (with one stage, the second's loads wrote zeros; they end before the wave does)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

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
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= ni) break;
#pragma unroll
      for (int v4 = 0; v4 < 4; ++v4) {
        f32x4_t quad[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int r = 0; r < 4; ++r) quad[q][r] = acc[i][q][4 * v4 + r];
        store_glu_quad(quad, bb, m0 + 64 * wm + 32 * i + 8 * v4 + 4 * fg, M, row0, ncol, N, lane,
                       reinterpret_cast<uint8_t*>(out), out_s, S);
      }
    }
  } else {
    if (ncol >= N) return;                                   // N % 32 == 0: four columns are all in or all out
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int m = m0 + 64 * wm + 32 * i + 8 * (v >> 2) + 4 * fg + (v & 3);
        if (m < M)
          *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + (size_t)(row0 + m) * N + ncol) =
              f32x4_t{acc[i][0][v] + bb[0], acc[i][1][v] + bb[1], acc[i][2][v] + bb[2], acc[i][3][v] + bb[3]};
      }
  }
}

// ---- the same product by tiles of 256 x 256 or 128 x 128 with K stages of 256 codes: a
// whole 128-byte line of every row and column at a time (with 64 bytes every load is a
// request to L2 of its own).  Two stage buffers of 68 or 34 KB: one workgroup of sixteen
// waves a CU, or two of four; each wave 64 x 64 = 4 x 4 blocks of
// v_mfma_scale_f32_16x16x128_f8f6f4, two steps of 128 values a stage.
//   LDS row 16j + t of a wave's 64 columns is column 4t + j, so a lane's four column
//   blocks are neighbouring columns, as in the tiles above; chunk c of row r sits at
//   slot c ^ ((r >> 1) & 7).
//   Lane (g = lane / 16, c = lane % 16) has block g of a step's four; its scales are
//   byte g of the row's word and the word of the four columns. ----
constexpr int kLine = 128;                         // bytes of a row and stage
template <int BM_, int BN_>
struct Lines {
  static constexpr int BM = BM_, BN = BN_, WN = BN / 64, WAVES = BM / 64 * WN, THREADS = WAVES * kWave;
  static constexpr int A = 0, B = A + BM * kLine, As = B + BN * kLine, Bs = As + 8 * BM, STAGE = Bs + 8 * BN;
  static constexpr int ALOADS = BM / 8 / WAVES, BLOADS = BN / 8 / WAVES;   // a wave and stage
  static constexpr int SA = BM / 32, SB = BN / 32, SLOADS = (SA + SB) / WAVES;   // loads of scales; of a wave
};

// one row block by four column blocks
__device__ __forceinline__ void products(f32x4_t (&acc)[4], u32x4_t a, const u32x4_t (&b)[4], uint32_t sa, uint32_t sb) {
  acc[0] = mfma_fp4_16<0, 0>(a, b[0], acc[0], sa, sb);
  acc[1] = mfma_fp4_16<0, 1>(a, b[1], acc[1], sa, sb);
  acc[2] = mfma_fp4_16<0, 2>(a, b[2], acc[2], sa, sb);
  acc[3] = mfma_fp4_16<0, 3>(a, b[3], acc[3], sa, sb);
}

template <bool GATE_UP, class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES == 16 ? 4 : 2) void w4a4_lines_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ As, const uint8_t* __restrict__ Wq,
    const uint8_t* __restrict__ Ws, const bf16_t* __restrict__ bias, const int32_t* __restrict__ cnt,
    const int32_t* __restrict__ off, const int32_t* __restrict__ rows, int K, int N, int E, int kslots, int a_rows,
    int64_t S, int n_tiles, void* __restrict__ out, uint8_t* __restrict__ out_s) {
  __shared__ __align__(1024) char smem_g[2 * C::STAGE];
  LDS3 char* smem = (LDS3 char*)smem_g;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int g = lane >> 4, c = lane & 15;

  int e, m0, nt;
  if (!grouped_gemm_tile(cnt, E, C::BM, n_tiles, kMBlock, lane, e, m0, nt)) return;   // workgroup-uniform
  const int n0 = nt * C::BN;
  const int M = cnt[e];
  // 256 rows: an expert's rows split evenly over its tiles, in steps of 64, which for two
  // tiles of up to 384 rows (three of up to 576) are tiles of 192; steps of 64 leave tiles
  // of 128 as they are
  int height = C::BM;
  if (C::BM > 128) {
    const int row_tiles = (M + C::BM - 1) / C::BM;
    height = (M + 64 * row_tiles - 1) / (64 * row_tiles) * 64;
    m0 = m0 / C::BM * height;
  }
  const int m_end = min(M, m0 + height);
  const int row0 = off[e];
  const int Kb = K / 2;
  const int nblk = K / 32;
  const int ns = (nblk + 7) / 8;

  // ---- direct-load assignments: each wave fills its share of the rows of A and of B,
  // eight an instruction (row 8i + l / 8, chunk (l % 8) ^ ((r >> 1) & 7)) ----
  const u32x4_t a_rs = rsrc_words(A, 0x7FFFFFFFu);
  const u32x4_t b_rs = rsrc_words(Wq + (size_t)e * N * Kb, 0x7FFFFFFFu);
  const u32x4_t as_rs = rsrc_words(As, 0x7FFFFFFFu);
  const u32x4_t bs_rs = rsrc_words(Ws + (size_t)e * nblk * N, 0x7FFFFFFFu);
  auto row_of = [&](int m) {
    return GATE_UP ? (uint32_t)(rows[row0 + m] / kslots) : (uint32_t)(row0 + m);
  };
  uint32_t a_off[C::ALOADS], b_off[C::BLOADS];
  auto row_a = [&](int i) { return C::BM / C::WAVES * wave + 8 * i + (lane >> 3); };
  auto row_b = [&](int i) { return C::BN / C::WAVES * wave + 8 * i + (lane >> 3); };
  auto chunk = [&](int r) { return (lane & 7) ^ ((r >> 1) & 7); };
#pragma unroll
  for (int i = 0; i < C::BLOADS; ++i) {
    const int r = row_b(i), n = n0 + (r & ~63) + 4 * (r & 15) + ((r >> 4) & 3);
    b_off[i] = n < N ? (uint32_t)n * (uint32_t)Kb + 16u * chunk(r) : kOOR;
  }
  // scales, 256 bytes an instruction: the first SA have 32 rows each (row l / 2, word l
  // % 2 of the stage's two), the others four columns a lane of one or two blocks
  uint32_t s_off[C::SLOADS];
  int s_blk[C::SLOADS];
  auto rows_scales = [&](int i) { return C::SLOADS == 2 ? i == 0 : wave < C::SA; };   // wave-uniform
  static_assert(C::SA == C::SB && (C::SLOADS == 1 || C::SLOADS == 2), "a wave has one load of each, or one");
#pragma unroll
  for (int i = 0; i < C::SLOADS; ++i) {
    const int at = 64 * (wave + C::WAVES * i - C::SA) + lane, n = n0 + at % (C::BN / 4) * 4;
    s_blk[i] = rows_scales(i) ? 4 * (lane & 1) : at / (C::BN / 4);
    s_off[i] = !rows_scales(i) && n < N ? (uint32_t)s_blk[i] * (uint32_t)N + (uint32_t)n : kOOR;
  }
  auto load_scales = [&](int i, int st, uint32_t at) {
    const uint32_t off = 8 * st + s_blk[i] < nblk ? s_off[i] : kOOR;
    if (rows_scales(i)) dma4(as_rs, off, (uint32_t)(2 * st) * (uint32_t)a_rows * 4u, at + C::As + 256 * (wave + C::WAVES * i));
    else dma4(bs_rs, off, (uint32_t)(8 * st) * (uint32_t)N, at + C::Bs + 256 * (wave + C::WAVES * i - C::SA));
  };
  auto load_b = [&](int st, int buf) {
    const uint32_t at = lds0 + buf * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::BLOADS; ++i)
      dma16(b_rs, 8 * st + chunk(row_b(i)) < nblk ? b_off[i] : kOOR, (uint32_t)st * kLine,
            at + C::B + (C::BN / C::WAVES * wave + 8 * i) * kLine);
  };
  auto load_a = [&](int st, int buf) {
    const uint32_t at = lds0 + buf * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::ALOADS; ++i)
      dma16(a_rs, 8 * st + chunk(row_a(i)) < nblk ? a_off[i] : kOOR, (uint32_t)st * kLine,
            at + C::A + (C::BM / C::WAVES * wave + 8 * i) * kLine);
#pragma unroll
    for (int i = 0; i < C::SLOADS; ++i) load_scales(i, st, at);
  };
  load_b(0, 0);   // ahead of the rows
#pragma unroll
  for (int i = 0; i < C::ALOADS; ++i) {
    const int m = m0 + row_a(i);
    a_off[i] = m < m_end ? row_of(m) * (uint32_t)Kb + 16u * chunk(row_a(i)) : kOOR;
  }
#pragma unroll
  for (int i = 0; i < C::SLOADS; ++i) {
    const int m = m0 + 32 * (wave + C::WAVES * i) + (lane >> 1);
    if (rows_scales(i) && m < m_end) s_off[i] = ((uint32_t)(lane & 1) * (uint32_t)a_rows + row_of(m)) * 4u;
  }
  load_a(0, 0);

  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const uint32_t xr = (uint32_t)((c >> 1) & 7);
  const uint32_t a_rd = C::A + (64 * wm + c) * kLine, b_rd = C::B + (64 * wn + c) * kLine;
  const bool live = m0 + 64 * wm < m_end;                      // wave-uniform: some of its rows are there
  for (int s = 0; s < ns; ++s) {
    const int buf = s & 1;
    // stage s has landed, and every wave is done with stage s - 1's buffer
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (s + 1 < ns) {
      load_b(s + 1, buf ^ 1);
      load_a(s + 1, buf ^ 1);
    }
    if (!live) continue;
    const LDS3 char* at = smem + buf * C::STAGE;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const bool in = 8 * s + 4 * t + g < nblk;            // no caller's byte past K is used: 255 would be a NaN
      const uint32_t xo = 16u * ((uint32_t)(4 * t + g) ^ xr);
      u32x4_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *(const LDS3 u32x4_t*)(at + b_rd + xo + 16 * j * kLine);
      const uint32_t sb = *(const LDS3 uint32_t*)(at + C::Bs + (4 * t + g) * C::BN + 64 * wn + 4 * c);
      if constexpr (C::WAVES == 4) {
        // all row blocks ahead of the products
        u32x4_t a[4];
        uint32_t sa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *(const LDS3 u32x4_t*)(at + a_rd + xo + 16 * i * kLine);
          sa[i] = *(const LDS3 uint8_t*)(at + C::As + 8 * (64 * wm + 16 * i + c) + 4 * t + g);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) products(acc[i], a[i], b, in ? sa[i] : 0u, sb);
      } else {
        // each before its own: four waves a SIMD have 128 registers each
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u32x4_t a = *(const LDS3 u32x4_t*)(at + a_rd + xo + 16 * i * kLine);
          const uint32_t sa = *(const LDS3 uint8_t*)(at + C::As + 8 * (64 * wm + 16 * i + c) + 4 * t + g);
          products(acc[i], a, b, in ? sa : 0u, sb);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  if (!live) return;

  // ---- epilogue: lane (g, c), element v of block (i, j): row 16i + 4g + v, column
  // 4c + j of the wave's 64 ----
  const int ncol = n0 + 64 * wn + 4 * c;
  float bb[4];
  {
    const uint32_t* bp = reinterpret_cast<const uint32_t*>(bias + (size_t)e * N + min(ncol, N - 4));
    const uint32_t b01 = bp[0], b23 = bp[1];
    bb[0] = bf16lo(b01), bb[1] = bf16hi(b01), bb[2] = bf16lo(b23), bb[3] = bf16hi(b23);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m4 = m0 + 64 * wm + 16 * i + 4 * g;          // rows m4 .. m4 + 3
    if constexpr (GATE_UP) {
      store_glu_quad(acc[i], bb, m4, m_end, row0, ncol, N, lane, reinterpret_cast<uint8_t*>(out), out_s, S);
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (m4 + v < m_end && ncol < N)
          *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + (size_t)(row0 + m4 + v) * N + ncol) =
              f32x4_t{acc[i][0][v] + bb[0], acc[i][1][v] + bb[1], acc[i][2][v] + bb[2], acc[i][3][v] + bb[3]};
    }
  }
}

template <bool GATE_UP>
hipError_t launch(const void* A, const void* As, const void* Wq, const void* Ws, const void* bias, const int32_t* cnt,
                  const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k, int64_t near,
                  void* out, void* out_s, hipStream_t stream) {
  const int64_t S = T * k, a_rows = GATE_UP ? T : S;
  // 32-bit buffer offsets: the token codes and one expert's codes below 2 GiB
  if (a_rows * K / 2 >= ((int64_t)1 << 31) || (int64_t)N * K / 2 >= ((int64_t)1 << 31)) return hipErrorNotSupported;
  // Three tilings by the mean rows an expert.  256 x 256 past 100, where it reads the
  // weights least often; for gate_up up to 250, since from there to some 800 rows two
  // workgroups a CU that multiply beside each other's GLU and codes are 2 to 7% ahead
  // (past 1000 they are 4 to 5% behind, with skewed picks of 128 experts 8%: one bound on
  // the mean does not follow that).  Up to 100, 128 x 128 where tiles of 128 x 256 are fewer
  // than 3.5 rounds of the 512 that run at a time (the last round is seldom full: 1288
  // of them are behind, 4416 ahead), else those.
  // gate_up (2880 x 5760) and down (2880 x 2880) in us, 128 x 256 | 128 x 128 | 256 x 256:
  //   32 experts, 64 rows each 100, 51 | 93, 50 | 94, 54;  96 rows 103, 56 | 97, 53 | 96,
  //   57;  128 rows 117, 77 | 126, 68 | 104, 62;  192 rows 131, 82 | 157, 79 | 116, 71;
  //   256 rows 172, 97 | 195, 105 | 172, 95;  313 rows 175, 112 | 213, 114 | 186, 91;
  //   512 rows 261, 170 | 319, 179 | 267, 154;  768 rows 355, 238 | 432, 253 | 370, 221;
  //   1024 rows 468, 309 | 599, 337 | 447, 284;  2048 rows 892, 562 | 1142, 636 | 855, 509;
  //   128 experts, 64 rows 312, 170 | 343, 171 | 355, 178;  104 rows 341, 207 | 377, 193 |
  //   385, 193;  128 rows 402, 235 | 467, 239 | 409, 205;  188 rows 484, 285 | 597, 299 |
  //   461, 237;  512 rows 1001, 619 | 1254, 676 | 1026, 581, skewed 1113, 713 | 1368, 732 |
  //   1026, 580.
  // Past 100 rows the number of tiles does not count, though few of them leave CUs idle: 8
  // experts of H = 1024, I = 512 with 128 or 256 rows, gate_up 15 and 14 us where 128 x
  // 128 takes 11; 16 experts of H = 4096, I = 1536 with 512 rows 92 where 256 x 256 takes 83.
  const int64_t wide = (near / kBM + (near < E ? near : E)) * ((N + kBN - 1) / kBN);
  auto run = [&](auto kern, int bm, int bn, int threads) {
    const int n_tiles = (N + bn - 1) / bn;
    // at most sum_e ceil(cnt_e / bm) <= S / bm + min(E, S) M tiles
    const int64_t tiles = (S / bm + (S < E ? S : E)) * n_tiles;
    const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(threads), 0, stream, (const uint8_t*)A, (const uint8_t*)As,
                       (const uint8_t*)Wq, (const uint8_t*)Ws, (const bf16_t*)bias, cnt, off, rows, K, N, E, k,
                       (int)a_rows, S, n_tiles, out, (uint8_t*)out_s);
    return hipGetLastError();
  };
  using Large = Lines<256, 256>;
  using Small = Lines<128, 128>;
  const bool many = near > 100 * (int64_t)E;
  if (many && (!GATE_UP || near <= 250 * (int64_t)E))
    return run(w4a4_lines_kernel<GATE_UP, Large>, Large::BM, Large::BN, Large::THREADS);
  if (!many && wide < 1792) return run(w4a4_lines_kernel<GATE_UP, Small>, Small::BM, Small::BN, Small::THREADS);
  return run(w4a4_gemm_kernel<GATE_UP>, kBM, kBN, kThreads);
}

}  // namespace

hipError_t launch_gemm_w4a4_gate_up(const void* xq, const void* sx, const void* Wq, const void* Ws, const void* bgu,
                                    const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                                    int k, int I, int64_t near, void* hq, void* sh, hipStream_t stream) {
  return launch<true>(xq, sx, Wq, Ws, bgu, cnt, off, rows, T, H, 2 * I, E, k, near, hq, sh, stream);
}

hipError_t launch_gemm_w4a4_down(const void* hq, const void* sh, const void* Wq, const void* Ws, const void* bd,
                                 const int32_t* cnt, const int32_t* off, int64_t T, int H, int E, int k, int I,
                                 int64_t near, float* o, hipStream_t stream) {
  return launch<false>(hq, sh, Wq, Ws, bd, cnt, off, nullptr, T, I, H, E, k, near, o, nullptr, stream);
}

}  // namespace moe
