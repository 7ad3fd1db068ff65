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
//        dw[s]     = sum over i of h d   (+ bd . dy)       in parts of 64 i
//   DX   dxs[s]    = dgu[s] . Wgu[e]^T                     [S][H]  (float32)
//   WGU  dWgu[e]   = sum over e's slots of x[t]^T dgu[s]   [H][2I] (bf16)
//   WD   dWd[e]    = sum over e's slots of wh[s]^T dy[t]   [I][H]  (bf16)
// 16 H I operations a slot.  dgu and wh are rounded to bf16 because they are
// operands of bf16 products, as h is in the forward pass; d stays float32, it
// is multiplied elementwise.
//
// One kernel for the five: tiles of 256 x 256, K stages of 64, four waves of 128
// x 128 = 4 x 4 blocks of v_mfma_f32_32x32x16_bf16.  An operand lies in memory
// either with K contiguous (rows of a stage are 128-byte lines) or with its rows
// or columns contiguous (a stage is 64 runs of 512 bytes, one for each k: Wgu in
// GU, all operands of the weight gradients, whose K is the expert's rows).  Both
// kinds go from HBM/L2 to LDS by direct loads of 16 bytes a lane, two stage
// buffers of 64 KB; fragments of the second kind are read by the transposing LDS
// read (ds_read_b64_tr_b16: 16 lanes read 4 k's x 16 columns and each gets the
// four k's of one column).
//   Tile heights: an expert's rows are split evenly over its tiles of at most 256,
//   in steps of 64, and a tile of 64 ni rows has ni row blocks a wave: the loop
//   is built for each ni.  530 rows cost three tiles of 192 and not of 256.
//   Stage layout, K contiguous: row r's 16-byte chunk c at slot c ^ ((r >> 1) &
//   7) of its 128 bytes.  Rows contiguous: run k's 32-byte piece p at p ^ 2 (k &
//   3) of its 512 bytes: the four k's of a transposing read fall on different
//   banks.
#include "device_common.h"
#include "launch.h"

#include <type_traits>

namespace moe {
namespace {

#define LDS3 __attribute__((address_space(3)))

typedef short s16x4_t __attribute__((ext_vector_type(4)));

enum Kind { kD, kGU, kDX, kWGU, kWD };

constexpr int kThreads = 256;
constexpr int kTile = 256;
constexpr int kBK = 64;
constexpr int kOpBytes = kTile * kBK * 2;   // 32 KB: one operand of one stage
constexpr int kA = 0;                       // A of buffer b at b * 32 KB
constexpr int kB = 2 * kOpBytes;            // B of buffer b at 64 KB + b * 32 KB
constexpr int kXcds = 8;
constexpr int kMBlock = 1024;               // M tiles per block of the tile order: all of an expert's
constexpr uint32_t kOOR = 0x80000000u;      // beyond every descriptor's range

struct Args {
  const bf16_t* A;
  const bf16_t* B;
  const int32_t *cnt, *off, *rows;
  int M, N, K;           // D, GU, DX: M unused; WGU, WD: K unused (the expert's rows)
  int E, kslots, tiles_m, tiles_n;
  void* out;
  // GU
  const bf16_t* bias;
  const float *d, *w;    // w [T][k]
  bf16_t* wh;
  float* dw_part;        // [ceil(2I / 128)][S]
  int64_t S;
};

__device__ __forceinline__ float xor1(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0xB1, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

template <int KIND>
__global__ __launch_bounds__(kThreads, 1) void backward_gemm_kernel(const Args p) {
  constexpr bool kWeightGrad = KIND == kWGU || KIND == kWD;
  constexpr bool kAT = kWeightGrad, kBT = kWeightGrad || KIND == kGU;   // rows / columns contiguous
  constexpr bool kAGather = KIND == kD || KIND == kGU || KIND == kWGU, kBGather = KIND == kWD;
  __shared__ __align__(1024) char smem_g[4 * kOpBytes];
  __shared__ float s_w[KIND == kGU ? kTile : 1];   // the rows' routing weights
  LDS3 char* smem = (LDS3 char*)smem_g;
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
    const int t = (int)(blockIdx.x % kXcds) * q + (int)blockIdx.x / kXcds;
    if ((int)blockIdx.x / kXcds >= q || t >= total) return;   // workgroup-uniform
    e = t / (p.tiles_m * p.tiles_n);
    const int r = t - e * p.tiles_m * p.tiles_n;
    nt = r / p.tiles_m;
    m0 = (r - nt * p.tiles_m) * kTile;
  } else {
    if (!grouped_gemm_tile(p.cnt, p.E, kTile, p.tiles_n, kMBlock, lane, e, m0, nt)) return;   // workgroup-uniform
  }
  const int n0 = nt * kTile;
  const int rows_e = p.cnt[e];
  const int row0 = p.off[e];
  const int M = kWeightGrad ? p.M : rows_e;
  const int K = kWeightGrad ? rows_e : p.K;
  const int N = p.N;
  const int ns = (K + kBK - 1) / kBK;
  // the tile's rows: an expert's split evenly over its tiles, in steps of 64
  int height = kTile;
  if (!kWeightGrad) {
    const int tiles = (M + kTile - 1) / kTile;
    height = (M + 64 * tiles - 1) / (64 * tiles) * 64;
    m0 = m0 / kTile * height;
  }
  const int m_end = min(M, m0 + height);
  const int ni = (m_end - m0 + 63) / 64;            // row blocks of 32 a wave, 1 .. 4
  if constexpr (KIND == kGU) {
    const int m = m0 + tid;
    s_w[tid] = m < m_end ? p.w[p.rows[row0 + m]] : 0.f;
  }

  // ---- direct-load assignments.  K contiguous: wave w fills rows 64w .. 64w +
  // 63, eight rows an instruction: lane l takes row 8i + l / 8 and the 16-byte
  // chunk (l % 8) ^ ((r >> 1) & 7).  Rows contiguous: wave w fills the runs of k
  // = 16w .. 16w + 15, two an instruction: lane l takes k = 16w + 2i + l / 32
  // and 16 bytes of piece ((l % 32) / 2) ^ 2 (k & 3).  What is past the edges is
  // sent out of range and lands as 0. ----
  const int lc[2] = {(lane & 7) ^ ((lane >> 4) & 7), (lane & 7) ^ (((lane >> 4) + 4) & 7)};   // even, odd i
  uint32_t a_off[8], b_off[8];
  u32x4_t a_rs, b_rs;
  uint32_t a_col[2], b_col[2];
  const bf16_t* Ae = p.A;
  const bf16_t* Be = p.B;
  if (!kAT) {
    // A rows: tokens' rows of dy or x, or the expert's rows of dgu from m0 on
    if (!kAGather) Ae += (size_t)(row0 + m0) * K;
    a_rs = rsrc_words(Ae, 0x7FFFFFFFu);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 64 * wave + 8 * i + (lane >> 3);
      const uint32_t c16 = 16u * (uint32_t)lc[i & 1];
      const uint32_t row = kAGather ? (uint32_t)(p.rows[row0 + min(m0 + r, M - 1)] / p.kslots) : (uint32_t)r;
      a_off[i] = m0 + r < m_end ? row * (uint32_t)K * 2u + c16 : kOOR;
    }
  }
  if (!kBT) {
    Be += (size_t)e * N * K;
    b_rs = rsrc_words(Be, 0x7FFFFFFFu);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = n0 + 64 * wave + 8 * i + (lane >> 3);
      b_off[i] = n < N ? (uint32_t)n * (uint32_t)K * 2u + 16u * (uint32_t)lc[i & 1] : kOOR;
    }
  }
  const int t_k = 16 * wave + (lane >> 5);          // k of instruction i: t_k + 2i
#pragma unroll
  for (int par = 0; par < 2; ++par) {
    const int f = 2 * ((2 * par + (lane >> 5)) & 3);
    const int col = 16 * (((lane & 31) >> 1) ^ f) + 8 * (lane & 1);
    a_col[par] = m0 + col < m_end ? 2u * (uint32_t)(m0 + col) : kOOR;
    b_col[par] = n0 + col < N ? 2u * (uint32_t)(n0 + col) : kOOR;
  }
  if (kBT && !kWeightGrad) Be += (size_t)e * N * K;                            // Wgu[e] [H][2I]
  if (kAT && !kAGather) Ae += (size_t)row0 * p.M;                              // wh of the expert's rows
  if (kWeightGrad && !kBGather) Be += (size_t)row0 * N;                        // dgu of the expert's rows

  // The tokens of the 16 k's that this wave loads at stage s (weight gradients)
  auto tokens = [&](int s) {
    const int k = s * kBK + 16 * wave + (lane & 15);
    return k < K ? (int)((uint32_t)p.rows[row0 + k] / (uint32_t)p.kslots) : 0;
  };
  int tok = 0, tok_next = 0;

  // one operand's instruction i of stage st
  auto dma_k = [&](u32x4_t rs, const uint32_t (&base)[8], int region, int st, int buf, int i) {
    const int k0 = st * kBK;
    const uint32_t voff = k0 + 8 * lc[i & 1] < K ? base[i] : kOOR;
    dma16(rs, voff, (uint32_t)k0 * 2u, lds0 + region + buf * kOpBytes + (64 * wave + 8 * i) * 128);
  };
  auto dma_t = [&](const bf16_t* base, int ld, const uint32_t (&col)[2], bool gather, int region, int st, int buf, int i) {
    const int k = st * kBK + t_k + 2 * i;
    uint32_t voff;
    u32x4_t rs;
    if (gather) {
      const int t0 = __builtin_amdgcn_readlane(tok, 2 * i), t1 = __builtin_amdgcn_readlane(tok, 2 * i + 1);
      voff = (uint32_t)(lane < 32 ? t0 : t1) * (uint32_t)ld * 2u + col[i & 1];
      rs = rsrc_words(base, 0x7FFFFFFFu);
    } else {
      voff = (uint32_t)(t_k + 2 * i) * (uint32_t)ld * 2u + col[i & 1];
      rs = rsrc_words(base + (size_t)st * kBK * ld, 0x7FFFFFFFu);
    }
    voff = k < K && col[i & 1] != kOOR ? voff : kOOR;
    dma16(rs, voff, 0u, lds0 + region + buf * kOpBytes + (16 * wave + 2 * i) * 512);
  };
  auto dma = [&](int st, int buf, int i, bool b_side) {
    if (b_side) {
      if constexpr (kBT) dma_t(Be, N, b_col, kBGather, kB, st, buf, i);
      else dma_k(b_rs, b_off, kB, st, buf, i);
    } else {
      if constexpr (kAT) dma_t(Ae, p.M, a_col, kAGather, kA, st, buf, i);
      else dma_k(a_rs, a_off, kA, st, buf, i);
    }
  };

  // ---- fragment reads: step j has k = 16j .. 16j + 15 of the stage ----
  const int fr = lane & 31, fg = lane >> 5;
  uint32_t a_rd[4], b_rd[4];   // K contiguous: of step j; rows contiguous: of fragment q
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t xo = 16u * (uint32_t)((2 * j + fg) ^ ((fr >> 1) & 7));
    const int r = (lane & 15) >> 2, half16 = (lane >> 4) & 1;
    const uint32_t run = (uint32_t)(8 * fg + r) * 512u + 8u * (uint32_t)(lane & 3);
    a_rd[j] = kAT ? (uint32_t)kA + run + 32u * (uint32_t)((2 * ni * wm + 2 * j + half16) ^ (2 * r))
                  : (uint32_t)(kA + (32 * ni * wm + fr) * 128) + xo;
    b_rd[j] = kBT ? (uint32_t)kB + run + 32u * (uint32_t)((8 * wn + 2 * j + half16) ^ (2 * r))
                  : (uint32_t)(kB + (128 * wn + fr) * 128) + xo;
  }
  auto read_t = [&](uint32_t at) -> u32x4_t {
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4_t*)(smem + at));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4_t*)(smem + at + 4 * 512));
    const u32x2_t l = __builtin_bit_cast(u32x2_t, lo), h = __builtin_bit_cast(u32x2_t, hi);
    return u32x4_t{l.x, l.y, h.x, h.y};
  };
  auto read_a = [&](int buf, int j, int q) -> u32x4_t {
    if constexpr (kAT) return read_t(a_rd[q] + buf * kOpBytes + j * 16 * 512);
    else return *(const LDS3 u32x4_t*)(smem + a_rd[j] + buf * kOpBytes + q * 32 * 128);
  };
  auto read_b = [&](int buf, int j, int q) -> u32x4_t {
    if constexpr (kBT) return read_t(b_rd[q] + buf * kOpBytes + j * 16 * 512);
    else return *(const LDS3 u32x4_t*)(smem + b_rd[j] + buf * kOpBytes + q * 32 * 128);
  };

  f32x16_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  // The loop for NI row blocks.  Step j of a stage in four slots: slot u reads row
  // fragment u (of the first NI) and column fragment u for step j and issues the
  // products of row block u of the step before; the slots of the first two steps
  // also issue the loads of stage s + 1 (past the last: none).
  auto loop = [&](auto ni_c) {
    constexpr int NI = decltype(ni_c)::value;
    u32x4_t fa0[4], fb0[4], fa1[4], fb1[4];
    auto multiply = [&](int u, const u32x4_t (&fa)[4], const u32x4_t (&fb)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[u][j] = mfma32x32x16(fa[u], fb[j], acc[u][j]);
    };
    auto step = [&](int s, int buf, int j, u32x4_t (&fa_rd)[4], u32x4_t (&fb_rd)[4], const u32x4_t (&fa_mm)[4],
                    const u32x4_t (&fb_mm)[4], bool do_mfma) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j < 2) {
          dma(s + 1, buf ^ 1, 4 * j + u, false);
          dma(s + 1, buf ^ 1, 4 * j + u, true);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (u < NI) fa_rd[u] = read_a(buf, j, u);
        fb_rd[u] = read_b(buf, j, u);
        if (u < NI && do_mfma) multiply(u, fa_mm, fb_mm);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int s = 0; s < ns; ++s) {
      const int buf = s & 1;
      if (kWeightGrad) {
        tok = tok_next;
        tok_next = tokens(s + 2);
      }
      step(s, buf, 0, fa0, fb0, fa1, fb1, s > 0);
      step(s, buf, 1, fa1, fb1, fa0, fb0, true);
      step(s, buf, 2, fa0, fb0, fa1, fb1, true);
      step(s, buf, 3, fa1, fb1, fa0, fb0, true);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
    }
#pragma unroll
    for (int u = 0; u < NI; ++u) multiply(u, fa1, fb1);
  };
  if (ns > 0) {
    // prologue: stage 0 into buffer 0
    if (kWeightGrad) {
      tok = tokens(0);
      tok_next = tokens(1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dma(0, 0, i, false);
      dma(0, 0, i, true);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (ni == 4) loop(std::integral_constant<int, 4>{});
    else if (ni == 3) loop(std::integral_constant<int, 3>{});
    else if (ni == 2) loop(std::integral_constant<int, 2>{});
    else loop(std::integral_constant<int, 1>{});
  }

  // ---- epilogue.  Lane l, element v of block (i, j): row 32i + 8 (v / 4) + 4 (l
  // / 32) + v % 4 of the wave's, column 32j + l % 32 of its 128.  Where a pair of
  // columns belongs together, lanes l and l ^ 1 exchange halves of two rows: the
  // even lane gets both columns of row v, the odd one those of row v + 1.
  // bf16 results go through LDS (the stage buffers are free behind the last
  // barrier), whose rows of 512 bytes then leave whole: 16-byte chunk c of row r
  // at c ^ 4 (r % 2 + 2 (r / 4 % 2)), as the four rows that a wave touches at once
  // would otherwise share their banks. ----
  const int row_w = 32 * ni * wm + 4 * fg;       // + 32 i + 8 (v / 4) + v % 4
  const bool odd = lane & 1;
  auto pair_of = [&](float v0, float v1, float& first, float& second) {
    const float got = xor1(odd ? v0 : v1);
    first = odd ? got : v0;
    second = odd ? v1 : got;
  };
  auto swizzle = [](int r) { return 4 * ((r & 1) + 2 * ((r >> 2) & 1)); };
  // word w (a pair of bf16, or a float) of row r: 128 words a row
  auto word_at = [&](int r, int w) { return (uint32_t)(r * 512 + 16 * ((w >> 2) ^ swizzle(r)) + 4 * (w & 3)); };
  // rows of 256 bf16 from LDS to out, which points at row m0, column n0
  auto flush = [&](bf16_t* out, int ld) {
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const int r = 64 * wave + 2 * i + (lane >> 5);
      const int c = 8 * ((lane & 31) ^ swizzle(r));
      const u32x4_t v = *(const LDS3 u32x4_t*)(smem + r * 512 + 16 * (lane & 31));
      if (m0 + r < m_end && n0 + c < N) *reinterpret_cast<u32x4_t*>(out + (size_t)r * ld + c) = v;
    }
  };
  if constexpr (KIND == kD || KIND == kDX) {
    float* out = reinterpret_cast<float*>(p.out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int m = m0 + row_w + 32 * i + 8 * (v >> 2) + (v & 3);
          if (m < m_end) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = n0 + 128 * wn + 32 * j + fr;
              if (n < N) out[(size_t)(row0 + m) * N + n] = acc[i][j][v];
            }
          }
        }
      }
    }
  } else if constexpr (kWeightGrad) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const int r = row_w + 32 * i + 8 * (v >> 2) + (v & 3) + (odd ? 1 : 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a, b;
            pair_of(acc[i][j][v], acc[i][j][v + 1], a, b);
            *(LDS3 uint32_t*)(smem + word_at(r, 64 * wn + 16 * j + (fr >> 1))) = pack_bf16x2(a, b);
          }
        }
      }
    }
    __syncthreads();
    flush(reinterpret_cast<bf16_t*>(p.out) + ((size_t)e * M + m0) * N + n0, N);
  } else {
    const int I = N / 2;
    // the tile of d: 256 rows x 128 floats, in the place that dgu takes
    {
      const u32x4_t d_rs = rsrc_words(p.d + (size_t)(row0 + m0) * I, 0x7FFFFFFFu);
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const int r = 64 * wave + 2 * i + (lane >> 5);
        const int c = n0 / 2 + 4 * ((lane & 31) ^ swizzle(r));
        dma16(d_rs, m0 + r < m_end && c < I ? ((uint32_t)r * (uint32_t)I + (uint32_t)c) * 4u : kOOR, 0u,
              lds0 + (64 * wave + 2 * i) * 512);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    }
    float bg[4], bu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + 128 * wn + 32 * j + (fr & ~1), N - 2);
      const uint32_t b = *reinterpret_cast<const uint32_t*>(p.bias + (size_t)e * N + n);
      bg[j] = bf16lo(b);
      bu[j] = bf16hi(b);
    }
    uint32_t wh[4][8][2];   // pairs j = 0, 1 and j = 2, 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const int r = row_w + 32 * i + 8 * (v >> 2) + (v & 3) + (odd ? 1 : 0);
          const float w = s_w[r];
          float dw = 0.f, whv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float gate, up;
            pair_of(acc[i][j][v], acc[i][j][v + 1], gate, up);
            gate += bg[j];
            up += bu[j];
            LDS3 uint32_t* at = (LDS3 uint32_t*)(smem + word_at(r, 64 * wn + 16 * j + (fr >> 1)));
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
    flush(reinterpret_cast<bf16_t*>(p.out) + (size_t)(row0 + m0) * N + n0, N);
    __syncthreads();
    // wh: rows of 128 bf16, 16-byte chunk c of row r at c ^ 2 (r % 2 + 2 (r / 4 % 2))
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < ni) {
#pragma unroll
        for (int v = 0; v < 16; v += 2) {
          const int r = row_w + 32 * i + 8 * (v >> 2) + (v & 3) + (odd ? 1 : 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = 64 * wn + 16 * j + (fr >> 1);
            *(LDS3 uint16_t*)(smem + r * 256 + 16 * ((c >> 3) ^ (swizzle(r) / 2)) + 2 * (c & 7)) =
                (uint16_t)(wh[i][v / 2][j / 2] >> (16 * (j & 1)));
          }
        }
      }
    }
    __syncthreads();
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
      const int r = 64 * wave + 4 * i + (lane >> 4);
      const int c = n0 / 2 + 8 * ((lane & 15) ^ (swizzle(r) / 2));
      const u32x4_t v = *(const LDS3 u32x4_t*)(smem + r * 256 + 16 * (lane & 15));
      if (m0 + r < m_end && c < I) *reinterpret_cast<u32x4_t*>(p.wh + (size_t)(row0 + m0 + r) * I + c) = v;
    }
  }
}

template <int KIND>
hipError_t launch(Args a, int64_t S, hipStream_t stream) {
  a.tiles_n = (a.N + kTile - 1) / kTile;
  int64_t tiles;
  if (KIND == kWGU || KIND == kWD) {
    a.tiles_m = (a.M + kTile - 1) / kTile;
    tiles = (int64_t)a.E * a.tiles_m * a.tiles_n;
  } else {
    // at most sum_e ceil(cnt_e / 256) <= S / 256 + min(E, S) tiles of rows
    tiles = (S / kTile + (S < a.E ? S : a.E)) * a.tiles_n;
  }
  const int64_t grid = (tiles + kXcds - 1) / kXcds * kXcds;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  a.S = S;
  hipLaunchKernelGGL((backward_gemm_kernel<KIND>), dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_backward_d(const void* dy, const void* Wd, const int32_t* cnt, const int32_t* off, const int32_t* rows,
                             int64_t T, int H, int E, int k, int I, float* d, hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)dy, a.B = (const bf16_t*)Wd, a.cnt = cnt, a.off = off, a.rows = rows;
  a.N = I, a.K = H, a.E = E, a.kslots = k, a.out = d;
  return launch<kD>(a, T * k, stream);
}

int backward_dw_parts(int I) { return (2 * I + kTile - 1) / kTile * 2; }

hipError_t launch_backward_gu(const void* x, const void* Wgu, const void* bgu, const float* w, const float* d,
                              const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                              int k, int I, void* dgu, void* wh, float* dw_part, hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)x, a.B = (const bf16_t*)Wgu, a.cnt = cnt, a.off = off, a.rows = rows;
  a.N = 2 * I, a.K = H, a.E = E, a.kslots = k, a.out = dgu;
  a.bias = (const bf16_t*)bgu, a.d = d, a.w = w, a.wh = (bf16_t*)wh, a.dw_part = dw_part;
  return launch<kGU>(a, T * k, stream);
}

hipError_t launch_backward_dx(const void* dgu, const void* Wgu, const int32_t* cnt, const int32_t* off, int64_t T, int H,
                              int E, int k, int I, float* dxs, hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)dgu, a.B = (const bf16_t*)Wgu, a.cnt = cnt, a.off = off;
  a.N = H, a.K = 2 * I, a.E = E, a.kslots = k, a.out = dxs;
  return launch<kDX>(a, T * k, stream);
}

hipError_t launch_backward_wgu(const void* x, const void* dgu, const int32_t* cnt, const int32_t* off,
                               const int32_t* rows, int64_t T, int H, int E, int k, int I, void* dWgu,
                               hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)x, a.B = (const bf16_t*)dgu, a.cnt = cnt, a.off = off, a.rows = rows;
  a.M = H, a.N = 2 * I, a.E = E, a.kslots = k, a.out = dWgu;
  return launch<kWGU>(a, T * k, stream);
}

hipError_t launch_backward_wd(const void* wh, const void* dy, const int32_t* cnt, const int32_t* off,
                              const int32_t* rows, int64_t T, int H, int E, int k, int I, void* dWd,
                              hipStream_t stream) {
  Args a{};
  a.A = (const bf16_t*)wh, a.B = (const bf16_t*)dy, a.cnt = cnt, a.off = off, a.rows = rows;
  a.M = I, a.N = H, a.E = E, a.kslots = k, a.out = dWd;
  return launch<kWD>(a, T * k, stream);
}

}  // namespace moe
