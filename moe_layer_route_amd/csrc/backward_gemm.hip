// Products of the block's backward pass: grouped GEMMs over the experts' rows
// (gradients of activations) and over the experts (gradients of weights).
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 2: per expert, gate_up ->
// bias -> clamped GLU -> down -> bias, weighted sum over the picks.  With dy the
// gradient of y, slot s = (token t, expert e, weight w), everything float32
// but the operands, which are bf16:
//   D    d[s]      = dy[t] . Wd[e]^T                       [S][I]  (float32)
//   GU   gate, up  = x[t] . Wgu[e] + bgu[e]                (recomputed)
//        g = min(gate, 7), u = clamp(up, -7, 7), z = sigmoid(1.702 g)
//        h = (u + 1) g z
//        dgu[s]    = w d * (dh/dgate, dh/dup)              [S][2I] (bf16)
//        wh[s]     = w h                                   [S][I]  (bf16)
//        dw[s]     = sum over i of h d   (+ bd . dy)       in parts of 48 i
//   DX   dxs[s]    = dgu[s] . Wgu[e]^T                     [S][H]  (float32)
//   WGU  dWgu[e]   = sum over e's slots of x[t]^T dgu[s]   [H][2I] (bf16)
//   WD   dWd[e]    = sum over e's slots of wh[s]^T dy[t]   [I][H]  (bf16)
// 16 H I operations a slot.  dgu and wh are rounded to bf16 because they are
// operands of bf16 products, as h is in the forward pass; d stays float32, it
// is multiplied elementwise.
//
// One kernel for the five: four waves in a 2 x 2 grid, each 64 rows x 96 or 128
// columns = 2 x 3 or 2 x 4 blocks of v_mfma_f32_32x32x16_bf16; two workgroups a CU,
// so that one's loads, exchange and stores run beside the other's products.
//   An operand lies in memory either with K contiguous or with its rows or columns
//   contiguous (a run for each k: Wgu in GU, both operands of the weight gradients,
//   whose K is the expert's rows).  Both kinds go from HBM/L2 to LDS by direct loads
//   of 16 bytes a lane; fragments of the second kind are read by the transposing LDS
//   read (ds_read_b64_tr_b16: 16 lanes read 4 k's x 16 columns and each gets the four
//   k's of one column).
//   D, GU, DX: tiles of 128 x 192, K stages of 64, a ring of two (80 KB).  A stage
//   has 128 bytes of a row: with stages of 32 every load of 64 bytes is a request to
//   L2 of its own (D of T = 4096, E = 32: 54 M requests and 392 us, against 29 M and
//   331).
//   WGU, WD: tiles of 128 x 256, K stages of 32, a ring of three (72 KB): runs are
//   whole lines anyway, an expert's rows are few stages, and the columns of the wider
//   tile are read by fewer of them (with 128 x 192 and 64: T = 4096 all gradients of
//   weights 1.25 -> 1.6 ms).
//   Measured against both and not kept: 256 x 256 by eight waves, one workgroup a CU,
//   stages of 64 (ring of two) or 32 (ring of four): the whole pass at T = 4096, E =
//   32 2.82 and 2.85 ms against 2.84, at T = 512 1.19 and 1.12 against 0.99.
//   An expert's last tile has what is left of its rows: with at most 64 a wave has
//   one row block instead of two.  The loop is built for either, and once more for the
//   tiles that reach past the last column, whose waves leave out the column blocks
//   without any.
// What bounds it (H = I = 2880, E = 32): at T = 4096, 512 rows an expert, the load
// path and the clock (1.9 to 2.0 GHz of 2.4): D 328 us (830 TFLOP/s), GU 673 (808), the
// rest 1.77 ms with the column sums (767), matrix pipes 38 to 46% busy.  Without the
// products they take 300, 603 and 1528 us, without the loads 203, 432 and 1123, without
// both 91, 227 and 618.  At T = 512, 64 rows, memory: D 105 us, GU 218, the rest 643 for
// 4.2 GB of weights read and gradients written, and without the products 105, 214, 605.
#include "backward_device.h"
#include "launch.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

#define LDS3 __attribute__((address_space(3)))

typedef short s16x4_t __attribute__((ext_vector_type(4)));

enum Kind { kD, kGU, kDX, kWGU, kWD };

constexpr int kThreads = 256;
constexpr int kBM = 128;

// The tile's columns, K stage and ring of a kind
template <int BN_, int BK_, int RING_, int PER_SLOT_>
struct Tile {
  static constexpr int BN = BN_, WN = BN / 2, NB = WN / 32;   // columns; of a wave; their blocks of 32
  static constexpr int BK = BK_, STEPS = BK / 16, WK = BK / 4;   // a stage's k's; of a wave's runs
  static constexpr int RING = RING_;                    // stage buffers; the loads run RING - 1 stages ahead
  static constexpr int PER_SLOT = PER_SLOT_;            // loads a slot of the loop
  static constexpr int ABYTES = kBM * BK * 2, BBYTES = BN * BK * 2;
  static constexpr int A = 0, B = RING * ABYTES;        // A and B of buffer b at b * ABYTES, b * BBYTES
  static constexpr int LDS = B + RING * BBYTES;
  static constexpr int ROW = BK * 2;                    // K contiguous: bytes of a row and stage
  static constexpr int RUN_A = kBM * 2, RUN_B = BN * 2; // rows contiguous: bytes of a run
  static constexpr int ALOADS = ABYTES / 4096, BLOADS = BBYTES / 4096;   // a wave and stage
};
template <int KIND>
using TileOf = std::conditional_t<KIND == kD || KIND == kDX || KIND == kGU, Tile<192, 64, 2, 4>, Tile<256, 32, 3, 1>>;
constexpr int kLds = 81920;                   // of the largest: two workgroups a CU
constexpr int kXcds = 8;
constexpr int kMBlock = 1024;               // M tiles per block of the tile order: all of an expert's
constexpr uint32_t kOOR = 0x80000000u;      // beyond every descriptor's range

struct Args {
  const bf16_t* A;
  const bf16_t* B;
  const int32_t *cnt, *off, *rows;
  int M, N, K;           // D, GU, DX: M unused; WGU, WD: K unused (the expert's rows)
  int E, tiles_m, tiles_n;
  uint32_t per_token;    // slot / k = umulhi(slot, per_token); 0: k = 1
  void* out;
  // GU
  const bf16_t* bias;
  const float *d, *w;    // w [T][k]
  bf16_t* wh;
  float* dw_part;        // [backward_dw_parts(I)][S]
  int64_t S;
};

__device__ __forceinline__ float xor1(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0xB1, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// One tile; block is the launch's number of it.
template <int KIND>
__device__ __forceinline__ void product(const Args& p, int block, LDS3 char* smem) {
  constexpr bool kWeightGrad = KIND == kWGU || KIND == kWD;
  using C = TileOf<KIND>;
  static_assert(C::LDS <= kLds, "two workgroups a CU");
  constexpr bool kAT = kWeightGrad, kBT = kWeightGrad || KIND == kGU;   // rows / columns contiguous
  constexpr bool kAGather = KIND == kD || KIND == kGU || KIND == kWGU, kBGather = KIND == kWD;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave >> 1, wn = wave & 1;

  // ---- workgroup -> expert and tile ----
  int e, m0, nt;
  if (kWeightGrad) {
    // consecutive tiles of an expert on one XCD
    const int total = p.E * p.tiles_m * p.tiles_n, q = (total + kXcds - 1) / kXcds;
    const int t = block % kXcds * q + block / kXcds;
    if (block / kXcds >= q || t >= total) return;   // workgroup-uniform
    e = t / (p.tiles_m * p.tiles_n);
    const int r = t - e * p.tiles_m * p.tiles_n;
    nt = r / p.tiles_m;
    m0 = (r - nt * p.tiles_m) * kBM;
  } else {
    // (these kinds come first in their launch: block is the workgroup's own number)
    if (!grouped_gemm_tile(p.cnt, p.E, kBM, p.tiles_n, kMBlock, lane, e, m0, nt)) return;   // workgroup-uniform
  }
  const int n0 = nt * C::BN;
  const int rows_e = p.cnt[e];
  const int row0 = p.off[e];
  const int M = kWeightGrad ? p.M : rows_e;
  const int K = kWeightGrad ? rows_e : p.K;
  const int N = p.N;
  const int ns = (K + C::BK - 1) / C::BK;
  const int m_end = min(M, m0 + kBM);
  const int ni = m_end - m0 > 64 ? 2 : 1;           // row blocks of 32 a wave
  auto token = [&](int slot) {
    return token_of((uint32_t)slot, p.per_token);
  };

  // ---- direct-load assignments.  K contiguous: wave w fills the w-th quarter of the
  // rows, 1 KB an instruction, a lane 16 bytes: chunk c of a row is at c ^ ((r >> 1)
  // & 7) of its 128 bytes.  Rows contiguous: wave w fills the w-th quarter of the
  // runs; 32-byte piece p of run k is at p ^ 2 (k & 3), in runs of 384 bytes, where
  // two k's are half the banks apart, at p ^ (k & 2): a transposing read's four k's
  // fall on different banks.  What is past the edges is sent out of range and lands
  // as 0. ----
  const bf16_t* Ae = p.A;
  const bf16_t* Be = p.B;
  auto row_i = [&](int i) { return 8 * i + (lane >> 3); };   // of the wave's rows
  auto chunk = [&](int i) { return (lane & 7) ^ ((row_i(i) >> 1) & 7); };
  static_assert(kWeightGrad || C::ROW == 128, "eight rows an instruction");
  constexpr int kRunChunksA = C::RUN_A / 16, kRunChunksB = C::RUN_B / 16;
  auto run_a = [&](int i) { return C::WK * wave + (64 * i + lane) / kRunChunksA; };
  auto run_b = [&](int i) { return C::WK * wave + (64 * i + lane) / kRunChunksB; };
  auto swizzle_b = [](int k) { return C::RUN_B == 512 ? 2 * (k & 3) : k & 2; };
  // of instruction i: K contiguous, the row's offset; rows contiguous, the column's
  uint32_t a_off[C::ALOADS], b_off[C::BLOADS];
#pragma unroll
  for (int i = 0; i < C::ALOADS; ++i) {
    if (kAT) {
      const int col = m0 + 16 * (((lane & 15) >> 1) ^ (2 * (run_a(i) & 3))) + 8 * (lane & 1);
      a_off[i] = col < m_end ? 2u * (uint32_t)col : kOOR;
    } else {
      const int m = m0 + kBM / 4 * wave + row_i(i);
      const uint32_t row = kAGather ? token(p.rows[row0 + min(m, M - 1)]) : (uint32_t)(m - m0);
      a_off[i] = m < m_end ? row * (uint32_t)K * 2u + 16u * (uint32_t)chunk(i) : kOOR;
    }
  }
#pragma unroll
  for (int i = 0; i < C::BLOADS; ++i) {
    if (kBT) {
      const int c = (64 * i + lane) % kRunChunksB;
      const int col = n0 + 16 * ((c >> 1) ^ swizzle_b(run_b(i))) + 8 * (c & 1);
      b_off[i] = col < N ? 2u * (uint32_t)col : kOOR;
    } else {
      const int n = n0 + C::BN / 4 * wave + row_i(i);
      b_off[i] = n < N ? (uint32_t)n * (uint32_t)K * 2u + 16u * (uint32_t)chunk(i) : kOOR;
    }
  }
  if (KIND == kDX) Ae += (size_t)(row0 + m0) * K;                              // dgu of the tile's rows
  if (kWeightGrad && !kAGather) Ae += (size_t)row0 * p.M;                      // wh of the expert's rows
  if (kWeightGrad && !kBGather) Be += (size_t)row0 * N;                        // dgu of the expert's rows
  if (!kWeightGrad) Be += (size_t)e * N * K;                                   // the expert's weight

  // The tokens of a wave's k's of a stage (weight gradients), loaded as scalars when
  // the stage before has been asked for: vector loads would be counted with the
  // direct loads, and the wait for them would drain those.  From the last row on, up
  // to WK - 1 words behind the expert's rows are read and not used.
  uint32_t tok[C::WK] = {};
  const __attribute__((address_space(4))) int32_t* const rows_s =
      (const __attribute__((address_space(4))) int32_t*)(p.rows + row0);
  auto tokens = [&](int s) {
    if constexpr (kWeightGrad) {
      const int k = min(s * C::BK + C::WK * wave, K - 1);
#pragma unroll
      for (int i = 0; i < C::WK; ++i) tok[i] = token(rows_s[k + i]);
    }
  };
  auto pick_a = [&](int i) {   // of the lane's k of A's instruction i: four runs
    const int g = lane >> 4;
    const uint32_t lo = g == 0 ? tok[4 * i] : tok[4 * i + 1], hi = g == 2 ? tok[4 * i + 2] : tok[4 * i + 3];
    return g < 2 ? lo : hi;
  };
  auto pick_b = [&](int i) { return lane < 32 ? tok[2 * i] : tok[2 * i + 1]; };   // of B's: two runs
  static_assert(!kWeightGrad || (C::RUN_A == 256 && C::RUN_B == 512), "the picks count the runs of an instruction");

  // load q of a wave's of stage st: A, then B
  auto load = [&](const bf16_t* base, int ld, bool t, bool gather, uint32_t off, int k_in, uint32_t token_row, int st,
                  uint32_t lds) {   // k_in: the first k in the stage of the lane's bytes
    const int k0 = st * C::BK;
    if (!t) {
      dma16(rsrc_words(base, 0x7FFFFFFFu), k0 + k_in < K ? off : kOOR, (uint32_t)k0 * 2u, lds);
    } else if (gather) {
      const uint32_t voff = token_row * (uint32_t)ld * 2u + off;
      dma16(rsrc_words(base, 0x7FFFFFFFu), k0 + k_in < K && off != kOOR ? voff : kOOR, 0u, lds);
    } else {
      const uint32_t voff = (uint32_t)k_in * (uint32_t)ld * 2u + off;
      dma16(rsrc_words(base + (size_t)k0 * ld, 0x7FFFFFFFu), k0 + k_in < K && off != kOOR ? voff : kOOR, 0u, lds);
    }
  };
  auto dma = [&](int st, int buf, int q) {
    if (q < C::ALOADS) {
      load(Ae, p.M, kAT, kAGather, a_off[q], kAT ? run_a(q) : 8 * chunk(q), kAT && kAGather ? pick_a(q) : 0u, st,
           lds0 + C::A + buf * C::ABYTES + wave * (C::ABYTES / 4) + 1024 * q);
    } else {
      const int i = q - C::ALOADS;
      load(Be, N, kBT, kBGather, b_off[i], kBT ? run_b(i) : 8 * chunk(i), kBT && kBGather ? pick_b(i) : 0u, st,
           lds0 + C::B + buf * C::BBYTES + wave * (C::BBYTES / 4) + 1024 * i);
    }
  };

  // ---- fragment reads: step j has k = 16j .. 16j + 15 of the stage ----
  const int fr = lane & 31, fg = lane >> 5;
  const int t_r = (lane & 15) >> 2, t_half = (lane >> 4) & 1;
  // K contiguous: of step 0, the others at ^ 32 j; rows contiguous: of fragment q
  uint32_t a_rd[2], b_rd[C::NB];
  const uint32_t xo = 16u * (uint32_t)(fg ^ ((fr >> 1) & 7));
#pragma unroll
  for (int q = 0; q < 2; ++q)
    a_rd[q] = kAT ? (uint32_t)(C::A + (8 * fg + t_r) * C::RUN_A + 8 * (lane & 3) +
                               32 * ((2 * ni * wm + 2 * q + t_half) ^ (2 * t_r)))
                  : (uint32_t)(C::A + (32 * ni * wm + fr) * C::ROW) + xo;
#pragma unroll
  for (int q = 0; q < C::NB; ++q)
    b_rd[q] = kBT ? (uint32_t)(C::B + (8 * fg + t_r) * C::RUN_B + 8 * (lane & 3) +
                               32 * ((C::WN / 16 * wn + 2 * q + t_half) ^ swizzle_b(t_r)))
                  : (uint32_t)(C::B + (C::WN * wn + fr) * C::ROW) + xo;
  auto read_t = [&](uint32_t at, int run) -> u32x4_t {
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4_t*)(smem + at));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4_t*)(smem + at + 4 * run));
    const u32x2_t l = __builtin_bit_cast(u32x2_t, lo), h = __builtin_bit_cast(u32x2_t, hi);
    return u32x4_t{l.x, l.y, h.x, h.y};
  };
  auto read_a = [&](int buf, int j, int q) -> u32x4_t {
    if constexpr (kAT) return read_t(a_rd[q] + buf * C::ABYTES + j * 16 * C::RUN_A, C::RUN_A);
    else return *(const LDS3 u32x4_t*)(smem + (a_rd[0] ^ (32 * j)) + buf * C::ABYTES + q * 32 * C::ROW);
  };
  auto read_b = [&](int buf, int j, int q) -> u32x4_t {
    if constexpr (kBT) return read_t(b_rd[q] + buf * C::BBYTES + j * 16 * C::RUN_B, C::RUN_B);
    else return *(const LDS3 u32x4_t*)(smem + (b_rd[0] ^ (32 * j)) + buf * C::BBYTES + q * 32 * C::ROW);
  };

  f32x16_t acc[2][C::NB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < C::NB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  // The loop for NI row blocks.  Step j of a stage in NB slots: slot u reads the
  // row fragment u (of the first NI) and the column fragment u for step j, issues
  // loads of the stage RING - 1 ahead, into the buffer that the stage before left at
  // the last barrier, and the products of column block u of the step before.
  // PART: only the first nj column blocks have columns.
  const int nj = min(C::NB, max(0, (N - n0 - C::WN * wn + 31) / 32));
  constexpr int kLoads = C::ALOADS + C::BLOADS;
  static_assert(C::RING == 2 || (C::RING == 3 && kLoads == 6), "the waits count the loads of a stage");
  static_assert(C::PER_SLOT * C::STEPS * C::NB >= kLoads, "every load has a slot");
  auto loop = [&](auto ni_c, auto part_c) {
    constexpr int NI = decltype(ni_c)::value;
    constexpr bool PART = decltype(part_c)::value;
    u32x4_t fa[2][2], fb[2][C::NB];
    auto multiply = [&](int u, int f) {
      if (PART && u >= nj) return;   // wave-uniform
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i][u] = mfma32x32x16(fa[f][i], fb[f][u], acc[i][u]);
    };
    int buf = 0, nbuf = C::RING - 1;
    for (int s = 0; s < ns; ++s) {
      const bool more = s + C::RING - 1 < ns;
#pragma unroll
      for (int j = 0; j < C::STEPS; ++j) {
#pragma unroll
        for (int u = 0; u < C::NB; ++u) {
          if (more) {
#pragma unroll
            for (int q = 0; q < C::PER_SLOT; ++q)
              if (C::PER_SLOT * (C::NB * j + u) + q < kLoads) dma(s + C::RING - 1, nbuf, C::PER_SLOT * (C::NB * j + u) + q);
          }
          __builtin_amdgcn_sched_barrier(0);
          if (u < NI) fa[j & 1][u] = read_a(buf, j, u);
          fb[j & 1][u] = read_b(buf, j, u);
          if (j > 0 || s > 0) multiply(u, (j & 1) ^ 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      tokens(s + C::RING);
      // stage s is read, and stage s + 1 has landed: with a ring of three when only the
      // loads of the stage behind it, if any, are out
      if (C::RING == 3 && more) asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      nbuf = buf;
      buf = buf == C::RING - 1 ? 0 : buf + 1;
    }
#pragma unroll
    for (int u = 0; u < C::NB; ++u) multiply(u, 1);
  };
  if (ns > 0) {
#pragma unroll
    for (int st = 0; st < C::RING - 1; ++st) {   // (out of range past the last stage)
      tokens(st);
#pragma unroll
      for (int q = 0; q < kLoads; ++q) dma(st, st, q);
    }
    tokens(C::RING - 1);
    if (C::RING == 3) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    using std::integral_constant;
    if (n0 + C::BN <= N) {
      if (ni == 2) loop(integral_constant<int, 2>{}, std::false_type{});
      else loop(integral_constant<int, 1>{}, std::false_type{});
    } else {
      if (ni == 2) loop(integral_constant<int, 2>{}, std::true_type{});
      else loop(integral_constant<int, 1>{}, std::true_type{});
    }
    __syncthreads();
  }

  // ---- epilogue.  Lane l, element v of block (i, j): row 32i + 8 (v / 4) + 4 (l
  // / 32) + v % 4 of the wave's, column 32j + l % 32 of its WN.  Where a pair of
  // columns belongs together, lanes l and l ^ 1 exchange halves of two rows: the
  // even lane gets both columns of row v, the odd one those of row v + 1.
  // GU's results go through LDS (the stage buffers are free behind the last
  // barrier), whose rows of 384 bytes then leave whole: 16-byte chunk c of row r at
  // c ^ (r & 4), as two of the four rows that a wave touches at once would otherwise
  // share their banks.  The weights' gradients leave from the registers, past the
  // caches (through LDS: the same time). ----
  const int row_w = 32 * ni * wm + 4 * fg;       // + 32 i + 8 (v / 4) + v % 4
  const bool odd = lane & 1;
  auto pair_of = [&](float v0, float v1, float& first, float& second) {
    const float got = xor1(odd ? v0 : v1);
    first = odd ? got : v0;
    second = odd ? v1 : got;
  };
  constexpr int kEpi = 2 * C::BN;                  // bytes of a row of d and of dgu
  // word w (a pair of bf16, or a float) of row r
  auto word_at = [&](int r, int w) { return (uint32_t)(r * kEpi + 16 * ((w >> 2) ^ (r & 4)) + 4 * (w & 3)); };
  if constexpr (KIND == kD || KIND == kDX) {
    float* out = reinterpret_cast<float*>(p.out);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int m = m0 + row_w + 32 * i + 8 * (v >> 2) + (v & 3);
          if (m < m_end) {
#pragma unroll
            for (int j = 0; j < C::NB; ++j) {
              const int n = n0 + C::WN * wn + 32 * j + fr;
              if (n < N) out[(size_t)(row0 + m) * N + n] = acc[i][j][v];
            }
          }
        }
      }
    }
  } else if constexpr (kWeightGrad) {
    // Of two column blocks j, j + 1 the even lane of a pair takes both columns of block
    // j, the odd one those of j + 1: an instruction stores whole lines, 64 columns of a
    // row.  Rows v and v + 1 are packed, so one exchange serves both.
    static_assert(C::NB % 2 == 0, "pairs of column blocks");
    const uint32_t pick_a = odd ? 0x01000504u : 0x05040100u, pick_b = odd ? 0x03020706u : 0x07060302u;
    const int col = C::WN * wn + (odd ? 32 : 0) + (fr & ~1);
    bf16_t* out = reinterpret_cast<bf16_t*>(p.out) + ((size_t)e * M + m0 + row_w) * N + n0 + col;
    const int rows_left = m_end - m0 - row_w, cols_left = N - n0 - col;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const int r = 32 * i + 8 * (v >> 2) + (v & 3);
          bf16_t* at = out + (size_t)r * N;
#pragma unroll
          for (int j = 0; j < C::NB; j += 2) {
            const uint32_t t0 = pack_bf16x2(acc[i][j][v], acc[i][j][v + 1]);
            const uint32_t t1 = pack_bf16x2(acc[i][j + 1][v], acc[i][j + 1][v + 1]);
            const uint32_t mine = odd ? t1 : t0;
            const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)(odd ? t0 : t1), 0xB1, 0xF, 0xF, true);
            if (32 * j < cols_left) {
              if (r < rows_left) __builtin_nontemporal_store(perm_b32(got, mine, pick_a), reinterpret_cast<uint32_t*>(at + 32 * j));
              if (r + 1 < rows_left)
                __builtin_nontemporal_store(perm_b32(got, mine, pick_b), reinterpret_cast<uint32_t*>(at + N + 32 * j));
            }
          }
        }
      }
    }
  } else {
    const int I = N / 2;
    constexpr int kChunks = kEpi / 16;
    static_assert(kBM * (kEpi + 4) <= kLds, "");
    LDS3 float* const s_w = (LDS3 float*)(smem + kBM * kEpi);
    // the tile of d, 128 rows x BN / 2 floats in the place that dgu takes, and the rows' weights
    {
      const u32x4_t d_rs = rsrc_words(p.d + (size_t)(row0 + m0) * I, 0x7FFFFFFFu);
#pragma unroll 6
      for (int i = 0; i < kChunks / 2; ++i) {
        const int at = 64 * (kChunks / 2 * wave + i) + lane, r = at / kChunks;
        const int c = n0 / 2 + 4 * ((at - r * kChunks) ^ (r & 4));
        dma16(d_rs, m0 + r < m_end && c < I ? ((uint32_t)r * (uint32_t)I + (uint32_t)c) * 4u : kOOR, 0u,
              lds0 + 1024 * (kChunks / 2 * wave + i));
      }
      if (tid < kBM) s_w[tid] = m0 + tid < m_end ? p.w[p.rows[row0 + m0 + tid]] : 0.f;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    }
    float bg[C::NB], bu[C::NB];
#pragma unroll
    for (int j = 0; j < C::NB; ++j) {
      const int n = min(n0 + C::WN * wn + 32 * j + (fr & ~1), N - 2);
      const uint32_t b = *reinterpret_cast<const uint32_t*>(p.bias + (size_t)e * N + n);
      bg[j] = bf16lo(b);
      bu[j] = bf16hi(b);
    }
    uint32_t wh[2][8][2];   // of two column blocks each
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const int r = row_w + 32 * i + 8 * (v >> 2) + (v & 3) + (odd ? 1 : 0);
          const float w = s_w[r];
          float dw = 0.f, whv[4] = {};
#pragma unroll
          for (int j = 0; j < C::NB; ++j) {
            float gate, up;
            pair_of(acc[i][j][v], acc[i][j][v + 1], gate, up);
            gate += bg[j];
            up += bu[j];
            LDS3 uint32_t* at = (LDS3 uint32_t*)(smem + word_at(r, C::WN / 2 * wn + 16 * j + (fr >> 1)));
            const float d = __uint_as_float(*at);   // 0 past the last row or column
            // compare-selects, so that a NaN stays one
            const float g = gate > 7.0f ? 7.0f : gate;
            const float u = up > 7.0f ? 7.0f : (up < -7.0f ? -7.0f : up);
            const float z = __builtin_amdgcn_rcpf(1.0f + __expf(-1.702f * g));
            const float gz = g * z;
            const float h = (u + 1.0f) * gz;
            dw = fmaf(h, d, dw);
            const float wd = w * d;
            const float dgate = gate > 7.0f ? 0.0f : wd * (u + 1.0f) * (z + 1.702f * gz * (1.0f - z));
            const float dup = up > 7.0f || up < -7.0f ? 0.0f : wd * gz;
            *at = pack_bf16x2(dgate, dup);
            whv[j] = w * h;
          }
          wh[i][v / 2][0] = pack_bf16x2(whv[0], whv[1]);
          wh[i][v / 2][1] = pack_bf16x2(whv[2], whv[3]);
          // lanes of one parity hold one row: sum over them, and over both halves of 32 lanes' columns
          dw = add_dpp<0x4E>(dw);    // quad_perm [2 3 0 1]
          dw = add_dpp<0x124>(dw);   // row_ror 4
          dw = add_dpp<0x128>(dw);   // row_ror 8
          dw += __shfl_xor(dw, 16, kWave);
          if (m0 + r < m_end && (lane & 30) == 0) p.dw_part[(size_t)(2 * nt + wn) * p.S + row0 + m0 + r] = dw;
        }
      }
    }
    __syncthreads();
    bf16_t* const dgu = reinterpret_cast<bf16_t*>(p.out) + (size_t)(row0 + m0) * N + n0;
#pragma unroll 6
    for (int i = 0; i < kChunks / 2; ++i) {
      const int at = kThreads * i + tid, r = at / kChunks, c = 8 * ((at - r * kChunks) ^ (r & 4));
      const u32x4_t v = *(const LDS3 u32x4_t*)(smem + 16 * at);
      if (m0 + r < m_end && n0 + c < N) *reinterpret_cast<u32x4_t*>(dgu + (size_t)r * N + c) = v;
    }
    __syncthreads();
    // wh: rows of BN / 2 bf16, 16-byte chunk c of row r at c ^ (r / 2 & 2)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const int r = row_w + 32 * i + 8 * (v >> 2) + (v & 3) + (odd ? 1 : 0);
#pragma unroll
          for (int j = 0; j < C::NB; ++j) {
            const int c = C::WN / 2 * wn + 16 * j + (fr >> 1);
            *(LDS3 uint16_t*)(smem + r * C::BN + 16 * ((c >> 3) ^ ((r >> 1) & 2)) + 2 * (c & 7)) =
                (uint16_t)(wh[i][v / 2][j / 2] >> (16 * (j & 1)));
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kChunks / 4; ++i) {
      const int at = kThreads * i + tid, r = at / (kChunks / 2);
      const int c = n0 / 2 + 8 * ((at - r * (kChunks / 2)) ^ ((r >> 1) & 2));
      const u32x4_t v = *(const LDS3 u32x4_t*)(smem + 16 * at);
      if (m0 + r < m_end && c < I) *reinterpret_cast<u32x4_t*>(p.wh + (size_t)(row0 + m0 + r) * I + c) = v;
    }
  }
}

template <int KIND>
__global__ __launch_bounds__(kThreads, 2) void backward_gemm_kernel(const Args p) {
  __shared__ __align__(1024) char smem[kLds];
  product<KIND>(p, blockIdx.x, (LDS3 char*)smem);
}

// What needs dgu and wh, in one launch: DX's tiles, which are long, the column sums and
// dl, then the tiles of the weight gradients, which are short and fill the places
// that DX's last round leaves (DX and others in turns: no gain; launches of their own:
// T = 512, E = 32 1155 -> 1080 us, T = 2047, E = 128 4257 -> 4059).  Blocks come in
// groups of eight, one a XCD.
struct Tail {
  Args dx, wgu, wd;
  Permuted slots;
  Sum dbgu, dbd;
  Dl dl;
  int begin[5];          // first group of the sums, dl, WGU, WD, and the end
};

__global__ __launch_bounds__(kThreads, 2) void backward_tail_kernel(const Tail p) {
  __shared__ __align__(1024) char smem_g[kLds];
  LDS3 char* smem = (LDS3 char*)smem_g;
  static_assert(kSumWaves * kWave == kThreads && kSumLds <= kLds, "column sums");
  const int group = blockIdx.x / kXcds;
  if (group < p.begin[0]) {
    product<kDX>(p.dx, blockIdx.x, smem);
  } else if (group < p.begin[1]) {
    const int item = blockIdx.x - p.begin[0] * kXcds, parts = p.dbgu.parts + p.dbd.parts;
    const int e = item / parts, piece = item - e * parts;
    if (e >= p.dx.E) return;                       // workgroup-uniform
    if (piece < p.dbgu.parts) column_sum<false>(p.dbgu, p.slots, e, piece, smem);
    else column_sum<true>(p.dbd, p.slots, e, piece - p.dbgu.parts, smem);
  } else if (group < p.begin[2]) {
    const int64_t t = (int64_t)(blockIdx.x - p.begin[1] * kXcds) * (kThreads / kWave) + threadIdx.x / kWave;
    if (t < p.dl.T) token_dl(p.dl, t, threadIdx.x & (kWave - 1));
  } else if (group < p.begin[3]) {
    product<kWGU>(p.wgu, blockIdx.x - p.begin[2] * kXcds, smem);
  } else {
    product<kWD>(p.wd, blockIdx.x - p.begin[3] * kXcds, smem);
  }
}

constexpr int64_t in_groups(int64_t blocks) { return (blocks + kXcds - 1) / kXcds; }

// groups of eight blocks of a product; fills in the tile counts
template <int KIND>
int64_t groups(Args& a, int64_t S) {
  constexpr int BN = TileOf<KIND>::BN;
  a.tiles_n = (a.N + BN - 1) / BN;
  int64_t tiles;
  if (KIND == kWGU || KIND == kWD) {
    a.tiles_m = (a.M + kBM - 1) / kBM;
    tiles = (int64_t)a.E * a.tiles_m * a.tiles_n;
  } else {
    // at most sum_e ceil(cnt_e / 128) <= S / 128 + min(E, S) tiles of rows
    tiles = (S / kBM + (S < a.E ? S : a.E)) * a.tiles_n;
  }
  a.S = S;
  return in_groups(tiles);
}

int64_t dl_groups(int64_t T) { return in_groups((T + kThreads / kWave - 1) / (kThreads / kWave)); }

template <int KIND>
hipError_t launch(Args a, int64_t S, hipStream_t stream) {
  const int64_t grid = groups<KIND>(a, S) * kXcds;
  hipLaunchKernelGGL((backward_gemm_kernel<KIND>), dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_backward_d(const void* dy, const void* Wd, const int32_t* cnt, const int32_t* off, const int32_t* rows,
                             int64_t T, int H, int E, int k, int I, float* d, hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)dy, a.B = (const bf16_t*)Wd, a.cnt = cnt, a.off = off, a.rows = rows;
  a.N = I, a.K = H, a.E = E, a.per_token = per_token(k), a.out = d;
  return launch<kD>(a, T * k, stream);
}

bool backward_fits(int64_t T, int H, int E, int k, int I) {
  const int64_t S = T * k;
  Args d{}, gu{}, dx{}, wgu{}, wd{};
  d.E = gu.E = dx.E = wgu.E = wd.E = E;
  d.N = I, gu.N = 2 * I, dx.N = H, wgu.M = H, wgu.N = 2 * I, wd.M = I, wd.N = H;
  const int64_t sums = (int64_t)E * ((2 * I + kSumCols - 1) / kSumCols + (H + kSumCols - 1) / kSumCols);
  const int64_t tail = groups<kDX>(dx, S) + in_groups(sums) + dl_groups(T) + groups<kWGU>(wgu, S) + groups<kWD>(wd, S);
  const int64_t most = std::max({groups<kD>(d, S), groups<kGU>(gu, S), tail});
  return most * kXcds * kThreads < (int64_t)1 << 32;
}

int backward_dw_parts(int I) {
  constexpr int BN = TileOf<kGU>::BN;
  return (2 * I + BN - 1) / BN * 2;
}

hipError_t launch_backward_gu(const void* x, const void* Wgu, const void* bgu, const float* w, const float* d,
                              const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                              int k, int I, void* dgu, void* wh, float* dw_part, hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)x, a.B = (const bf16_t*)Wgu, a.cnt = cnt, a.off = off, a.rows = rows;
  a.N = 2 * I, a.K = H, a.E = E, a.per_token = per_token(k), a.out = dgu;
  a.bias = (const bf16_t*)bgu, a.d = d, a.w = w, a.wh = (bf16_t*)wh, a.dw_part = dw_part;
  return launch<kGU>(a, T * k, stream);
}

hipError_t launch_backward_tail(const void* dy, const void* x, const void* Wgu, const void* bd, const int32_t* ids,
                                const float* w, const float* dw_part, const void* dgu, const void* wh,
                                const int32_t* cnt, const int32_t* off, const int32_t* rows, const int32_t* pos,
                                int64_t T, int H, int E, int k, int I, float* dxs, float* dl, void* dWgu, void* dbgu,
                                void* dWd, void* dbd, hipStream_t stream) {
  const int64_t S = T * k;
  Tail p{};
  Args a{};
  a.cnt = cnt, a.off = off, a.rows = rows, a.E = E, a.per_token = per_token(k);
  p.dx = p.wgu = p.wd = a;
  p.dx.A = (const bf16_t*)dgu, p.dx.B = (const bf16_t*)Wgu, p.dx.N = H, p.dx.K = 2 * I, p.dx.out = dxs;
  p.wgu.A = (const bf16_t*)x, p.wgu.B = (const bf16_t*)dgu, p.wgu.M = H, p.wgu.N = 2 * I, p.wgu.out = dWgu;
  p.wd.A = (const bf16_t*)wh, p.wd.B = (const bf16_t*)dy, p.wd.M = I, p.wd.N = H, p.wd.out = dWd;
  p.slots = Permuted{cnt, off, rows, a.per_token};
  p.dbgu = sum_of(dgu, nullptr, 2 * I, dbgu, nullptr);
  p.dbd = sum_of(dy, w, H, dbd, nullptr);
  p.dl = Dl{(const bf16_t*)dy, (const bf16_t*)bd, ids, pos, w, dw_part, backward_dw_parts(I), H, k, T, dl};
  const int64_t n[5] = {groups<kDX>(p.dx, S), in_groups((int64_t)E * (p.dbgu.parts + p.dbd.parts)), dl_groups(T),
                        dWgu ? groups<kWGU>(p.wgu, S) : 0, dWd ? groups<kWD>(p.wd, S) : 0};
  int64_t at = 0;
  for (int i = 0; i < 5; ++i) p.begin[i] = (int)(at += n[i]);
  hipLaunchKernelGGL(backward_tail_kernel, dim3((unsigned)(at * kXcds)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace moe
