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
#include "int4_device.h"
#include "few_slots.h"
#include "launch.h"
#include "route_key.h"
#include "wave_reduce.h"

#include <type_traits>

namespace moe {
namespace {

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

// ---------------------------------------------------------------------------
// Quantiser: one thread per (column, group).  Symmetric: s = bf16(max|v| / 7),
// q = clamp(rint(v / s), -8, 7) + 8.  With zero points: lo = min(v, 0),
// hi = max(v, 0), s = bf16(hi / 15 - lo / 15), z = clamp(rint(-lo / s), 0,
// 15), q = clamp(rint(v / s) + z, 0, 15).  float32, halves to even; s = 0
// gives q = z (and z = 0 with zero points).  Run once when weights are loaded: 32
// experts of 2880 x 5760 take 1.02 ms at G = 64, 1.05 at G = 128 with zero points,
// 1.3 TB/s of the weights, codes and scales.
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
// thread per stored word, which is four consecutive source bytes.  32 experts of
// 2880 x 5760 take 0.32 ms, 1.7 TB/s: a tile reads 16 bytes of each of 64 columns.
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
// Weight streaming: a workgroup owns one expert and one strip of 64 columns;
// its WAVES waves split K and stream their part of the strip, a contiguous
// kilobyte a tile, four tiles (a quad, 128 values of K) at a time and one quad
// ahead.  16 MG token rows per pass over the strip.
//   Operands of v_mfma_f32_16x16x32_bf16: A = 16 token rows, lane (row c,
//   group g) holding K = 32 kt + 8 g .. + 7; B = word j of the tile, i.e. MFMA
//   column c of call j is column 4 c + j of the strip, so the four columns of
//   a lane are two (gate, up) pairs.
//   NS strips share the token rows' loads: rows cost as many bytes of the
//   path from L2 into a CU as the 64 columns they meet, and twice as many with
//   two chunks (T = 192 of 32 experts, 24 rows each: 90 us with one strip, 74
//   with two).
//   A word gives 16 + q exactly (seven integer instructions for eight codes).
//   The 16 and the zero point come off through the accumulator: a group's sum
//   starts at -(16 + z) sum(a), where sum(a) is one more MFMA with a constant
//   operand (-24 without zero points, 1 with them).  The group's sum times its
//   scale is added to the accumulators in float32.
// What binds is HBM: T = 64 of 32 experts, 2880 x 5760, G = 64 with zero points
// 51.3 us, 5.7 TB/s of the 6.1 that a plain read of as much reaches; T = 256 of
// 128 experts, 2880 x 2880, G = 128 95.3 us, 5.9 TB/s; T = 8 of 32 experts, G =
// 32 33.1 us, 5.9 TB/s.
// ---------------------------------------------------------------------------
constexpr int kCus = 256;

// The n-th expert that has rows (in order; E <= 256): its index, row count and
// first row.  Every lane gets the same; false if there are fewer.
__device__ __forceinline__ bool nth_live_expert(const int32_t* __restrict__ cnt, const int32_t* __restrict__ off, int E,
                                                int n, int lane, int& e, int& M, int& row0) {
  int c[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = kWave * i + lane;
    c[i] = at < E ? cnt[at] : 0;
    o[i] = at < E ? off[at] : 0;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t live = __ballot(c[i] > 0);
    const int here = __popcll(live);
    if (n < here) {
      const int rank = __popcll(live & ((1ull << lane) - 1));
      const int src = __ffsll((unsigned long long)__ballot(c[i] > 0 && rank == n)) - 1;
      e = kWave * i + src;
      M = __builtin_amdgcn_readlane(c[i], src);
      row0 = __builtin_amdgcn_readlane(o[i], src);
      return true;
    }
    n -= here;
  }
  return false;
}

// Where a workgroup's expert and rows come from:
//   kGrouped  the permutation: expert blockIdx.y, or the n-th one that has rows;
//   kSlots    one token slot each (blockIdx.y = k t + j), for few tokens: gate_up
//             picks the slot's expert from the router's logits (every wave by
//             itself, which costs it less than a launch), and one more column of
//             workgroups writes the decision for the later launches; down reads
//             it.  Two slots of one expert read its weights twice.
enum Mode { kGrouped, kSlots };

template <bool GATE_UP, int MG, int GS, bool ZERO, int WAVES, int NS, Mode MODE>
__global__ __launch_bounds__(WAVES * kWave, WAVES == 8 || MG > 1 || NS > GS ? 2 : 3) void int4_stream_kernel(
    const bf16_t* __restrict__ A, const uint8_t* __restrict__ Wq, const uint16_t* __restrict__ Ws,
    const uint8_t* __restrict__ Wz, const bf16_t* __restrict__ bias, const int32_t* __restrict__ cnt,
    const int32_t* __restrict__ off, const int32_t* __restrict__ rows, int K, int N, int E, int kslots,
    int64_t a_rows, void* __restrict__ out, Slots slots) {
  constexpr int NGQ = 4 / GS;
  __shared__ float red[WAVES][4][4][kWave];   // [wave][call j][element v][lane]

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int strips = (N + kTileN - 1) / kTileN;
  int e = blockIdx.y, M, row0;
  if (MODE == kSlots) {
    M = 1, row0 = blockIdx.y;
    if (GATE_UP) {
      const int t = (int)blockIdx.y / slots.k, j = (int)blockIdx.y % slots.k;
      const bool decide = (int)blockIdx.x * NS >= strips;   // block-uniform: past the strips
      if (decide && (j != 0 || wave != 0)) return;          // no barrier follows there
      if (decide) return write_decision(slots, t, E, lane);
      e = slot_expert(slots, t, j, E, lane);
    } else {
      e = slots.ids[blockIdx.y];
    }
  } else if ((int)gridDim.y == E) {
    M = cnt[e], row0 = off[e];
    if (M == 0) return;   // block-uniform
  } else if (!nth_live_expert(cnt, off, E, blockIdx.y, lane, e, M, row0)) {
    return;               // block-uniform
  }
  const int g = lane >> 4, c = lane & 15;
  const int nkt = K / kTileK, nq = (nkt + 3) / 4, ng = (nkt + GS - 1) / GS;
  // N % 8 == 0: a lane's four columns of a strip are all in range or all out
  int ncol[NS];
  uint32_t s_col[NS];
  const uint8_t* w_base[NS];
  uint32_t b01[NS], b23[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const int strip = blockIdx.x * NS + n;
    ncol[n] = strip * kTileN + 4 * c;
    s_col[n] = (uint32_t)min(ncol[n], N - 4);
    w_base[n] = Wq + ((size_t)e * strips + min(strip, strips - 1)) * (size_t)nkt * kTileBytes;
    const uint32_t* bp = reinterpret_cast<const uint32_t*>(bias + (size_t)e * N + s_col[n]);   // 4-byte aligned
    b01[n] = bp[0], b23[n] = bp[1];
  }
  const bf16_t* a_base = GATE_UP ? A : A + (size_t)row0 * K;
  const uint32_t a_bytes = (uint32_t)((size_t)(GATE_UP ? a_rows : M) * K * 2);
  const int q_begin = nq * wave / WAVES, q_end = nq * (wave + 1) / WAVES;
  const int kt_end = min(nkt, 4 * q_end);
  const u32x4_t flat = ZERO ? u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}
                            : u32x4_t{0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};
  const Int4Masks masks;

  for (int r0 = 0; r0 < M; r0 += 16 * MG) {
    const int nch = min(MG, (M - r0 + 15) / 16);   // block-uniform
    int slot[MG];
#pragma unroll
    for (int m = 0; m < MG; ++m) {
      const int r = min(r0 + 16 * m + c, M - 1);   // rows past M repeat the last one
      slot[m] = !GATE_UP ? r : MODE == kSlots ? row0 : rows[row0 + r];
    }
    f32x4_t acc[NS][MG][4];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int m = 0; m < MG; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Tile kt's codes and rows; one that is not there (past K, or past the wave's
    // share) reads nothing and gives zeros.
    u32x4_t w[NS][4], a[MG][4];
    auto load_w = [&](int n, int t, int kt) __attribute__((always_inline)) {
      w[n][t] = buf_ld16<2>(make_rsrc(w_base[n], kt < kt_end ? nkt * kTileBytes : 0), 16u * lane,
                               (uint32_t)kt * kTileBytes);   // read once
    };
    uint32_t a_off[MG];
    auto load_a = [&](int t, int kt) __attribute__((always_inline)) {
      const rsrc_t a_rs = make_rsrc(a_base, kt < kt_end ? a_bytes : 0u);
#pragma unroll
      for (int m = 0; m < MG; ++m) a[m][t] = buf_ld16(a_rs, a_off[m], 64u * (uint32_t)kt);
    };
    u32x2_t s[NS][NGQ];
    uint32_t z[NS][NGQ];
    auto load_s = [&](int q) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NGQ; ++i) {
        // a group past K has the scale 0
        const bool in = NGQ * q + i < ng;
        const rsrc_t s_rs = make_rsrc(Ws + (size_t)e * ng * N, in ? (uint32_t)ng * N * 2 : 0u);
        const uint32_t at = (uint32_t)(NGQ * q + i) * N;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          s[n][i] = __builtin_bit_cast(
              u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(s_rs, (int)(2u * s_col[n]), (int)(2u * at), 0));
          if (ZERO)
            z[n][i] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(Wz + (size_t)e * ng * N, in ? (uint32_t)ng * N : 0u),
                                                           (int)s_col[n], (int)at, 0);
        }
      }
    };
    // One quad's products; each tile's registers are refilled with the next
    // quad's as soon as its last product has read them.
    auto quad = [&](auto more, int q) __attribute__((always_inline)) {
      constexpr bool kMore = decltype(more)::value;
      u32x2_t sq[NS][NGQ];
      uint32_t zq[NS][NGQ];
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < NGQ; ++i) {
          sq[n][i] = s[n][i];
          if (ZERO) zq[n][i] = z[n][i];
        }
      if (kMore) load_s(q + 1);
#pragma unroll
      for (int i = 0; i < NGQ; ++i) {
        f32x4_t sum[MG];
#pragma unroll
        for (int m = 0; m < MG; ++m) {
          sum[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int t = GS * i; t < GS * i + GS; ++t) sum[m] = mfma16x16x32(a[m][t], flat, sum[m]);
        }
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          // one group of one strip after the other (below, its sums are added
          // at once): the compiler would otherwise keep all partial sums to the end
          __builtin_amdgcn_sched_barrier(0);
          float sf[4], zf[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sf[j] = j & 1 ? bf16hi(sq[n][i][j >> 1]) : bf16lo(sq[n][i][j >> 1]);
            if (ZERO) zf[j] = -16.0f - (float)((zq[n][i] >> (8 * j)) & 0xFFu);
          }
          f32x4_t part[MG][4];
#pragma unroll
          for (int m = 0; m < MG; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v) part[m][j][v] = ZERO ? zf[j] * sum[m][v] : sum[m][v];
#pragma unroll
          for (int t = GS * i; t < GS * i + GS; ++t) {
            __builtin_amdgcn_sched_barrier(0);   // tile by tile, or the operands of all of them fill the registers
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const u32x4_t bw = int4_operand(w[n][t][j], masks);
#pragma unroll
              for (int m = 0; m < MG; ++m) part[m][j] = mfma16x16x32(a[m][t], bw, part[m][j]);
            }
            if (kMore) load_w(n, t, 4 * q + 4 + t);
            if (kMore && n == NS - 1) load_a(t, 4 * q + 4 + t);
          }
#pragma unroll
          for (int m = 0; m < MG; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[n][m][j][v] = __builtin_fmaf(sf[j], part[m][j][v], acc[n][m][j][v]);
              asm volatile("" : "+v"(acc[n][m][j]));
            }
        }
      }
    };

    if (q_begin < q_end) {
      // The weights are under way while the rows' slots arrive.
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NS; ++n) load_w(n, t, 4 * q_begin + t);
      load_s(q_begin);
#pragma unroll
      for (int m = 0; m < MG; ++m)
        a_off[m] = ((uint32_t)(GATE_UP ? slot[m] / kslots : slot[m]) * (uint32_t)K + 8u * g) * 2u;
#pragma unroll
      for (int t = 0; t < 4; ++t) load_a(t, 4 * q_begin + t);
      int q = q_begin;
      for (; q + 1 < q_end; ++q) quad(std::true_type{}, q);
      quad(std::false_type{}, q);
    }

    // Sum the K partials in the waves' order; wave w < 4 finishes element v = w
    // (row 4 g + w of each chunk) of the lane's four columns.
#pragma unroll
    for (int m = 0; m < MG; ++m) {
#pragma unroll
     for (int n = 0; n < NS; ++n) {
      if (m < nch) {
        const float bb[4] = {bf16lo(b01[n]), bf16hi(b01[n]), bf16lo(b23[n]), bf16hi(b23[n])};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) red[wave][j][v][lane] = acc[n][m][j][v];
        __syncthreads();
        const int r = r0 + 16 * m + 4 * g + wave;
        if (wave < 4 && r < M && ncol[n] < N) {
          float sum[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float t = 0.f;
#pragma unroll
            for (int w2 = 0; w2 < WAVES; ++w2) t += red[w2][j][wave & 3][lane];
            sum[j] = t + bb[j];
          }
          const size_t orow = (size_t)(row0 + r);
          if (GATE_UP)
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(out) + orow * (N / 2) + ncol[n] / 2) =
                pack_bf16x2(clamped_glu(sum[0], sum[1]), clamped_glu(sum[2], sum[3]));
          else
            *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + orow * N + ncol[n]) =
                f32x4_t{sum[0], sum[1], sum[2], sum[3]};
        }
        __syncthreads();
      }
     }
    }
  }
}

template <bool GATE_UP, int MG, int GS, int WAVES, int NS, Mode MODE>
hipError_t launch_stream(const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias,
                         const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E,
                         int k, int experts, void* out, const Slots& slots, hipStream_t stream) {
  const int columns = ((N + kTileN - 1) / kTileN + NS - 1) / NS;
  dim3 grid((unsigned)(columns + (MODE == kSlots && GATE_UP ? 1 : 0)), (unsigned)experts);
  auto kern = Wz ? int4_stream_kernel<GATE_UP, MG, GS, true, WAVES, NS, MODE>
                 : int4_stream_kernel<GATE_UP, MG, GS, false, WAVES, NS, MODE>;
  hipLaunchKernelGGL(kern, grid, dim3(WAVES * kWave), 0, stream, (const bf16_t*)A, (const uint8_t*)Wq,
                     (const uint16_t*)Ws, (const uint8_t*)Wz, (const bf16_t*)bias, cnt, off, rows, K, N, E, k, T, out,
                     slots);
  return hipGetLastError();
}

template <bool GATE_UP, int MG, int WAVES, int NS, Mode MODE>
hipError_t launch_group(int G, const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias,
                        const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E,
                        int k, int experts, void* out, const Slots& slots, hipStream_t stream) {
  auto launch = G == 32   ? launch_stream<GATE_UP, MG, 1, WAVES, NS, MODE>
                : G == 64 ? launch_stream<GATE_UP, MG, 2, WAVES, NS, MODE>
                          : launch_stream<GATE_UP, MG, 4, WAVES, NS, MODE>;
  return launch(A, Wq, Ws, Wz, bias, cnt, off, rows, T, K, N, E, k, experts, out, slots, stream);
}

// Mean rows per expert up to which one 16-row chunk a pass is enough, and from
// which most experts have rows, so that two strips a wave still leave every CU
// two workgroups where the grid has them.  (T = 8, 32, 64 of 32 experts, 2880
// columns and more: gate_up with one strip 33.6, 47.0, 53.5 us, with two 36.6,
// 46.5, 52.3; T = 256 of 128 experts: down 104 against 98.6 us.  64 rows of 32
// experts of 1024 x 1536, 384 workgroups of two strips: 8.8 against 10.3 us.)
// On an expert-parallel rank T * k is the whole layer's and E the rank's: the mean
// is taken E_layer / E times too high there, and both switches come earlier than
// the rank's own rows call for.
// Where no CU would get a second workgroup, eight waves halve each one's share
// of K.
constexpr int64_t kOneChunkMeanRows = 10;
constexpr int64_t kTwoStripsMeanRows = 4;

template <bool GATE_UP>
hipError_t launch_int4(const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias,
                       const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k,
                       int G, void* out, hipStream_t stream) {
  // 32-bit offsets into the token rows (of one expert, for down)
  if ((GATE_UP ? T : T * k) * K * 2 >= (int64_t)1 << 32) return hipErrorNotSupported;
  // No more experts than slots have rows: with fewer slots than experts the
  // workgroups go to the ones that have.
  const int experts = (int)(T * k < E ? T * k : E);
  const int64_t workgroups = (int64_t)experts * ((N + kTileN - 1) / kTileN);
  const bool two = T * k >= kTwoStripsMeanRows * E && workgroups >= 4 * kCus;
  auto launch = T * k > kOneChunkMeanRows * E
                    ? (two ? launch_group<GATE_UP, 2, 4, 2, kGrouped> : launch_group<GATE_UP, 2, 4, 1, kGrouped>)
                : two                ? launch_group<GATE_UP, 1, 4, 2, kGrouped>
                : workgroups <= kCus ? launch_group<GATE_UP, 1, 8, 1, kGrouped>
                                     : launch_group<GATE_UP, 1, 4, 1, kGrouped>;
  return launch(G, A, Wq, Ws, Wz, bias, cnt, off, rows, T, K, N, E, k, experts, out, Slots{}, stream);
}

// One workgroup column per token slot (the rows of h and o in slot order).
template <bool GATE_UP>
hipError_t launch_slots(const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias, int64_t T, int K,
                        int N, int E, int G, void* out, const Slots& slots, hipStream_t stream) {
  const int S = (int)T * slots.k;
  const int64_t workgroups = (int64_t)S * ((N + kTileN - 1) / kTileN);
  auto launch = workgroups <= kCus ? launch_group<GATE_UP, 1, 8, 1, kSlots> : launch_group<GATE_UP, 1, 4, 1, kSlots>;
  return launch(G, A, Wq, Ws, Wz, bias, nullptr, nullptr, nullptr, GATE_UP ? T : S, K, N, E, slots.k, S, out, slots, stream);
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

hipError_t launch_int4_slots(const void* x, const void* Wr, const void* br, const void* Wgu_q, const void* Wgu_s,
                             const void* Wgu_z, const void* bgu, const void* Wd_q, const void* Wd_s, const void* Wd_z,
                             const void* bd, int64_t T, int H, int E, int k, int I, int G, double* logits, int32_t* ids,
                             float* w, int32_t* pos, void* h, float* o, hipStream_t stream) {
  hipError_t e = launch_few_logits(x, Wr, br, T, H, E, logits, stream);
  if (e != hipSuccess) return e;
  const Slots slots{logits, ids, w, pos, k};
  e = launch_slots<true>(x, Wgu_q, Wgu_s, Wgu_z, bgu, T, H, 2 * I, E, G, h, slots, stream);
  if (e != hipSuccess) return e;
  return launch_slots<false>(h, Wd_q, Wd_s, Wd_z, bd, T, I, H, E, G, o, slots, stream);
}

hipError_t launch_int4_gate_up(const void* x, const void* Wq, const void* Ws, const void* Wz, const void* bgu,
                               const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int H, int E,
                               int k, int I, int G, void* h, hipStream_t stream) {
  return launch_int4<true>(x, Wq, Ws, Wz, bgu, cnt, off, rows, T, H, 2 * I, E, k, G, h, stream);
}

hipError_t launch_int4_down(const void* h, const void* Wq, const void* Ws, const void* Wz, const void* bd,
                            const int32_t* cnt, const int32_t* off, int64_t T, int H, int E, int k, int I, int G, float* o,
                            hipStream_t stream) {
  return launch_int4<false>(h, Wq, Ws, Wz, bd, cnt, off, nullptr, T, I, H, E, k, G, o, stream);
}

}  // namespace moe
