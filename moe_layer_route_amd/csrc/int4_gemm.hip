// Grouped GEMMs of the experts with 4-bit integer weights (many rows per
// expert).
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 5 (one batched launch for
// all experts, 4-bit weights) and section 2 (gate_up -> bias -> GLU, down ->
// bias).  The format and the exact 16 + q operands are those of int4.hip.
//
// A workgroup owns 128 rows x 512 columns of one expert: eight waves, two per
// SIMD, each with a strip of 64 columns (128 accumulators a lane) and all 128
// rows; or, where there are few tiles, half of each with four waves, two
// workgroups on a CU.  K goes in units of GU tiles that never cross a group of the scales
// (64 values, or 32 where the groups are of 32).  A unit's token rows come into
// LDS by direct loads, fragment by fragment (a fragment is the 16-row operand
// of one MFMA, a kilobyte), two or three units ahead in a ring of four, and so
// do the wave's own tiles of weights, their scales and zero points.  (Weights loaded
// into registers: 873 against 774 us at the first size below.  The compiler
// counts only the loads it makes itself, so its waits for them take in the
// direct loads under way.)  Per 16-row chunk the unit's products go into a
// fresh accumulator that starts at -(16 + z) sum(a) and is added to the result,
// times the scale, in float32: no weight is rounded.  A unit of two tiles and
// 64 products has 198 vector instructions beside them: 128 of these additions
// (zero points: 128 multiplications more), 56 to unpack the codes, 14 for
// addresses.
//
// T = 4096 of 32 experts, 2880 x 5760 (gate_up), G = 64: 570 us, 954 TFLOP/s;
// down 324 us, 839 TFLOP/s (a large library product reaches 1155 to 1300 here);
// T = 16384: 2113 us, 1029 TFLOP/s.  No unit is saturated: at T = 4096 the matrix
// pipes are busy for 45% of the cycles (down 38%), vector instructions and
// products issue in 54% (42%), the LDS is busy for 22%; a wave waits for a load
// or a barrier for 26% of its time (30%) and for its turn to issue for 30%.  Two
// waves a SIMD, which is all that 128 accumulators a lane leave room for, do not
// cover each other's waits.
#include "device_common.h"
#include "int4_device.h"
#include "launch.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kRing = 4;
constexpr int kXcds = 8;
constexpr int kMBlock = 8;   // M tiles that take an N tile together
constexpr uint32_t kOutOfRange = 0xFFFFFFF0u;

template <int GU, int W>
struct Ring {
  u32x4_t rows[kRing][GU][W][kWave];   // fragments of the token rows, in lane order
  u32x4_t w[W][kRing][GU][kWave];      // each wave's tiles
  uint32_t s[W][kRing][kWave];         // scales of its 64 columns, twice
  uint32_t z[W][kRing][kWave];         // zero points, four times
  float sum[4][W][16];                          // of each row's values over a unit, times `flat`
};

// Which tile a workgroup takes.  An expert has ceil(M / kBM) M tiles x n_tiles N
// tiles.  They come in three rounds, the long ones first, so that the last to
// run are short (T = 1024: 128 rows an expert on average, and every second one
// has a tile of a few rows: gate_up 244 us in one sequence, 195 in rounds):
//   0  M tiles with more than kBM / 2 rows x the `wide` N tiles whose strips are
//      all there: expert by expert, kMBlock M tiles taking each N tile in turn;
//   1  an expert's shorter last M tile x those N tiles;
//   2  every M tile x the N tile that is not `wide`.
// A round's tiles are dealt to the XCDs (block b runs on XCD b % 8) in equal
// consecutive parts, whose L2 serves the tiles that share rows or weights.
// Every lane gets the same; false for a block past the last tile (the grid is an
// upper bound).  Lane l counts experts 4 l .. 4 l + 3: E <= 256.
template <int kBM>
__device__ __forceinline__ bool tile_of(const int32_t* __restrict__ cnt, int E, int n_tiles, int wide, int lane, int& e,
                                        int& m0, int& nt) {
  int longer[4], shorter[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = lane * 4 + i, M = at < E ? cnt[at] : 0, rest = M % kBM;
    longer[i] = M / kBM + (rest > kBM / 2);
    shorter[i] = rest > 0 && rest <= kBM / 2;
  }
  int xi = (int)blockIdx.x / kXcds;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int cols = round < 2 ? wide : n_tiles - wide;
    int tiles[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tiles[i] = ((round != 1 ? longer[i] : 0) + (round != 0 ? shorter[i] : 0)) * cols;
      sum += tiles[i];
    }
    const int incl = wave_incl_scan(sum, lane);
    const int all = __builtin_amdgcn_readlane(incl, kWave - 1), share = (all + kXcds - 1) / kXcds;
    if (xi >= share) {   // block-uniform
      xi -= share;
      continue;
    }
    const int at = (int)(blockIdx.x % kXcds) * share + xi;
    if (at >= all) return false;
    int fe = -1, fm = 0, fn = 0, start = incl - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at >= start && at < start + tiles[i]) {
        const int t = at - start;
        fe = lane * 4 + i;
        if (round == 0) {
          const int block = t / (kMBlock * wide), in_block = t - block * kMBlock * wide;
          const int height = min(kMBlock, longer[i] - block * kMBlock);
          fm = block * kMBlock + in_block % height, fn = in_block / height;
        } else if (round == 1) {
          fm = longer[i], fn = t;
        } else {
          fm = t, fn = wide;
        }
      }
      start += tiles[i];
    }
    const int src = __ffsll((unsigned long long)__ballot(fe >= 0)) - 1;
    e = __builtin_amdgcn_readlane(fe, src);
    m0 = __builtin_amdgcn_readlane(fm, src) * kBM;
    nt = __builtin_amdgcn_readlane(fn, src);
    return true;
  }
  return false;
}

template <bool GATE_UP, int GU, bool ZERO, int W>
__global__ __launch_bounds__(W * kWave, 2) void int4_gemm_kernel(
    const bf16_t* __restrict__ A, const uint8_t* __restrict__ Wq, const uint16_t* __restrict__ Ws,
    const uint8_t* __restrict__ Wz, const bf16_t* __restrict__ bias, const int32_t* __restrict__ cnt,
    const int32_t* __restrict__ off, const int32_t* __restrict__ rows, int K, int N, int E, int kslots, int64_t a_rows,
    int n_tiles, int units_per_group, void* __restrict__ out) {
  static_assert(W == 4 || W == 8, "a wave brings in one chunk; run() below counts them");
  constexpr int kChunks = W, kBM = 16 * kChunks;
  // Two workgroups of four waves on a CU run out of step by themselves; of eight
  // waves the second half is shifted (below) where the registers allow it, which
  // costs a unit of the ring.
  constexpr bool kShift = W == 8 && !(ZERO && GU == 2);
  constexpr int kAhead = kShift ? 2 : 3;
  __shared__ __align__(16) Ring<GU, W> ring;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int e, m0, nt;
  if (!tile_of<kBM>(cnt, E, n_tiles, (N + kTileN - 1) / kTileN / W, lane, e, m0, nt)) return;   // block-uniform
  const int M = cnt[e], row0 = off[e];
  const int nch = min(kChunks, (M - m0 + 15) / 16);   // chunks with rows
  const int g = lane >> 4, c = lane & 15;
  const int nkt = K / kTileK, nu = (nkt + GU - 1) / GU;
  const int ng = (nu + units_per_group - 1) / units_per_group;
  const int strips = (N + kTileN - 1) / kTileN;
  const int strip = nt * W + wave;
  const bool live = strip < strips;   // wave-uniform; a wave past the last strip only loads rows
  const int ncol = strip * kTileN + 4 * c;
  const int wstrip = min(strip, strips - 1);

  const u32x4_t w_rs = rsrc_words(Wq + ((size_t)e * strips + wstrip) * (size_t)nkt * kTileBytes, (uint32_t)nkt * kTileBytes);
  const u32x4_t s_rs = rsrc_words(Ws + (size_t)e * ng * N, (uint32_t)ng * N * 2);
  const u32x4_t z_rs = rsrc_words(ZERO ? Wz + (size_t)e * ng * N : Wq, ZERO ? (uint32_t)ng * N : 0u);
  const u32x4_t a_rs = rsrc_words(GATE_UP ? A : A + (size_t)row0 * K, (uint32_t)((size_t)(GATE_UP ? a_rows : M) * K * 2));

  // wave w brings in chunk w's fragments: lane (row c, group g); rows past M
  // repeat the last one, a chunk without rows reads nothing (zeros), columns
  // past N are the last ones
  const int r = min(m0 + 16 * wave + c, M - 1);
  const uint32_t a_off = m0 + 16 * wave >= M ? kOutOfRange
                                             : ((uint32_t)(GATE_UP ? rows[row0 + r] / kslots : r) * (uint32_t)K +
                                                8u * g) * 2u;
  const uint32_t s_off = 2u * (uint32_t)min(wstrip * kTileN + 2 * (lane & 31), N - 2);
  const uint32_t z_off = (uint32_t)min(wstrip * kTileN + 4 * c, N - 4);
  const uint32_t rows_at = (uint32_t)(uintptr_t)&ring.rows[0][0][wave][0];
  const uint32_t w_at = (uint32_t)(uintptr_t)&ring.w[wave][0][0][0];
  const uint32_t s_at = (uint32_t)(uintptr_t)&ring.s[wave][0][0], z_at = (uint32_t)(uintptr_t)&ring.z[wave][0][0];
  // Every wave issues the same loads for every unit, past the end too (where
  // nothing is read): the waits count on it.
  constexpr int kLoads = 2 * GU + 1 + (ZERO ? 1 : 0);
  auto load = [&](int u, int i) __attribute__((always_inline)) {
    const int slot = u % kRing;
    if (i < 2 * GU) {
      const int t = i >> 1, kt = GU * u + t;
      const bool in = kt < nkt;
      if ((i & 1) == 0)
        dma16(a_rs, in ? a_off : kOutOfRange, in ? 64u * (uint32_t)kt : 0u,
              rows_at + (uint32_t)((slot * GU + t) * kChunks * kWave) * 16u);
      else
        dma16(w_rs, in ? 16u * (uint32_t)lane : kOutOfRange, in ? (uint32_t)kt * kTileBytes : 0u,
              w_at + (uint32_t)((slot * GU + t) * kWave) * 16u);
    } else {
      const uint32_t at = (uint32_t)(min(u, nu - 1) / units_per_group) * N;
      if (i == 2 * GU)
        dma4(s_rs, s_off, 2u * at, s_at + (uint32_t)(slot * kWave) * 4u);
      else
        dma4(z_rs, z_off, at, z_at + (uint32_t)(slot * kWave) * 4u);
    }
  };
  auto load_all = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(u, i);
  };
  const u32x4_t flat = ZERO ? u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}
                            : u32x4_t{0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};
  f32x4_t acc[kChunks][4];
#pragma unroll
  for (int m = 0; m < kChunks; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // A unit's codes, scales and zero points of this lane.
  struct Words {
    u32x4_t w[GU];
    u32x2_t s;
    uint32_t z;
  };
  auto words = [&](int u, Words& b) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < GU; ++t) b.w[t] = ring.w[wave][u % kRing][t][lane];
    b.s = *reinterpret_cast<const u32x2_t*>(&ring.s[wave][u % kRing][2 * c]);
    if (ZERO) b.z = ring.z[wave][u % kRing][c];
  };
  // The chunk's operands from LDS.
  auto chunk_in = [&](int u, int m, u32x4_t (&a)[GU]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < GU; ++t) a[t] = ring.rows[u % kRing][t][m][lane];
  };
  // Unit u's sums over the rows of this wave's own chunk (whose fragments the
  // wave itself brought in), for all waves behind the next barrier: one more
  // product with a constant operand, the same in every column.
  auto sum_rows = [&](int u) __attribute__((always_inline)) {
    u32x4_t a[GU];
    chunk_in(u, wave, a);
    f32x4_t sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < GU; ++t) sum = mfma16x16x32(a[t], flat, sum);
    if (c == 0) *reinterpret_cast<f32x4_t*>(&ring.sum[u & 3][wave][4 * g]) = sum;
  };
  auto sum_in = [&](int u, int m) __attribute__((always_inline)) {
    return *reinterpret_cast<const f32x4_t*>(&ring.sum[u & 3][m][4 * g]);
  };
  auto chunk_mul = [&](const u32x4_t (&a)[GU], const f32x4_t& sum, const u32x4_t (&bw)[GU][4], const float (&z)[4],
                       f32x4_t (&part)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[j][v] = ZERO ? z[j] * sum[v] : sum[v];
#pragma unroll
    for (int t = 0; t < GU; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[j] = mfma16x16x32(a[t], bw[t][j], part[j]);
  };
  auto chunk_add = [&](f32x4_t (&sums)[4], const f32x4_t (&part)[4], const float (&s)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int v = 0; v < 4; ++v) sums[j][v] = __builtin_fmaf(s[j], part[j][v], sums[j][v]);
      asm volatile("" : "+v"(sums[j]));   // here, not at the end: the parts would fill the registers
    }
  };
  const Int4Masks masks;
  // What a wave prepares of the next unit: loads retire in order, so with those
  // of the units behind it still under way its own part of unit u is in LDS.
  auto next = [&](int u) __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * kLoads) : "memory");
    sum_rows(u);
  };
  auto compute = [&](auto count, auto shift, int u, const Words& b) __attribute__((always_inline)) {
    float s[4], z[4];
    u32x4_t bw[GU][4];
#pragma unroll
    for (int t = 0; t < GU; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) bw[t][j] = int4_operand(b.w[t][j], masks);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = j & 1 ? bf16hi(b.s[j >> 1]) : bf16lo(b.s[j >> 1]);
      if (ZERO) z[j] = -16.0f - (float)((b.z >> (8 * j)) & 0xFFu);
    }
    // Without branches: a chunk is read two ahead of its products and added
    // behind the next one's.
    constexpr int kCount = decltype(count)::value, kHalf = kCount / 2;
    constexpr bool kLate = decltype(shift)::value;
    u32x4_t a[3][GU];
    f32x4_t sum[3], part[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      chunk_in(u, m, a[m]);
      sum[m] = sum_in(u, m);
    }
#pragma unroll
    for (int m = 0; m < kCount; ++m) {
      __builtin_amdgcn_sched_barrier(0);
      // The loads of the unit kAhead ahead (one more for the second half of a
      // late wave's unit, which is past the barrier), into the slot that every
      // wave has left; spread over the chunks: a load that the CU's load path
      // cannot take yet holds up its wave's products.
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (kLate ? kHalf + i * kHalf / kLoads == m : i * (kCount - 1) / kLoads == m) load(kLate ? u + kAhead + 1 : u + kAhead, i);
      if (m + 2 < kCount) {
        chunk_in(u, m + 2, a[(m + 2) % 3]);
        sum[(m + 2) % 3] = sum_in(u, m + 2);
      }
      chunk_mul(a[m % 3], sum[m % 3], bw, z, part[m & 1]);
      if (m == (kLate ? kHalf : kCount) - 1) {
        next(u + 1);
        if (kLate) __syncthreads();
      }
      if (m > 0) chunk_add(acc[m - 1], part[(m - 1) & 1], s);
    }
    chunk_add(acc[kCount - 1], part[(kCount - 1) & 1], s);
  };

  // Every SIMD has one wave of each half of the workgroup.  The second half runs
  // half a unit behind: its barriers stand in the middle of a unit, so that one
  // wave unpacks its weights, and waits, while the other has products to issue
  // (T = 4096, G = 64: 595 us in step, 570 like this; with zero points and units
  // of two tiles it takes 14 registers too many).
  const bool late = kShift && live && wave >= W / 2;
  for (int u = 0; u < kAhead; ++u) load_all(u);
  Words b;
  next(0);
  words(0, b);
  if (late) load_all(kAhead);
  __syncthreads();
  // The wave's own weights it may read at once, the other waves' rows and sums
  // behind the barrier.  Barrier u stands behind the first waves' unit u and
  // amid the late ones' (which have read unit u - 1 by then): with late waves the
  // slots of u - 1, u and u + 1 are in use between barriers u - 1 and u, and the
  // loads of u + 2 go to the fourth; without, u, u + 1 and u + 2, and u + 3.
  auto run = [&](auto count) __attribute__((always_inline)) {
    if (late) {
      for (int u = 0; u < nu; ++u) {
        compute(count, std::true_type{}, u, b);
        words(u + 1, b);
      }
    } else {
      for (int u = 0; u < nu; ++u) {
        if (live) {
          compute(count, std::false_type{}, u, b);
        } else {
          load_all(u + kAhead);
          next(u + 1);
        }
        words(u + 1, b);
        __syncthreads();
      }
    }
  };
  // an even count of chunks: at most one is computed for nothing
  if (W == 8 && nch > 6)
    run(std::integral_constant<int, W>{});
  else if (W == 8 && nch > 4)
    run(std::integral_constant<int, W == 8 ? 6 : 4>{});
  else if (nch > 2)
    run(std::integral_constant<int, 4>{});
  else
    run(std::integral_constant<int, 2>{});
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may reach this LDS after the workgroup's end
  if (!live || ncol >= N) return;                    // no barrier follows

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

template <bool GATE_UP, int W>
hipError_t launch_tiles(const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias,
                        const int32_t* cnt, const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k,
                        int G, void* out, hipStream_t stream) {
  const int n_tiles = (N + W * kTileN - 1) / (W * kTileN);
  const int64_t m_slots = (T * k + 16 * W - 1) / (16 * W) + E;
  // tile_of rounds each of its three rounds up to the XCDs
  const int64_t grid = (n_tiles * m_slots + 3 * (kXcds - 1) + kXcds - 1) / kXcds * kXcds;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = G == 32 ? (Wz ? int4_gemm_kernel<GATE_UP, 1, true, W> : int4_gemm_kernel<GATE_UP, 1, false, W>)
                      : (Wz ? int4_gemm_kernel<GATE_UP, 2, true, W> : int4_gemm_kernel<GATE_UP, 2, false, W>);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(W * kWave), 0, stream, (const bf16_t*)A, (const uint8_t*)Wq,
                     (const uint16_t*)Ws, (const uint8_t*)Wz, (const bf16_t*)bias, cnt, off, rows, K, N, E, k, T, n_tiles,
                     G == 128 ? 2 : 1, out);
  return hipGetLastError();
}

// Two workgroups of small tiles fit a CU.  Where all of them run at once they
// are done sooner than fewer CUs with large ones, which unpack each weight for
// half as many rows (K = 2048, N = 4096, G = 64, 104 rows an expert: 8 experts
// 33 against 56 us, 16 42 against 57, 32, more than fit at once, 88 against 79).
// Eight rows more than the mean are counted: an expert past 64 has one tile more.
// An expert-parallel rank passes the whole layer's T * k with its own E, which
// counts the layer's rows for the local experts: it takes the large tiles earlier
// than its own rows call for.
constexpr int64_t kSmallTiles = 512;

template <bool GATE_UP>
hipError_t launch(const void* A, const void* Wq, const void* Ws, const void* Wz, const void* bias, const int32_t* cnt,
                  const int32_t* off, const int32_t* rows, int64_t T, int K, int N, int E, int k, int G, void* out,
                  hipStream_t stream) {
  const int64_t S = T * k;
  // 32-bit offsets into the token rows (of one expert, for down)
  if ((GATE_UP ? T : S) * K * 2 >= (int64_t)1 << 32) return hipErrorNotSupported;
  const int64_t small = (N + 4 * kTileN - 1) / (4 * kTileN) * ((S + 72 * (int64_t)E - 1) / (64 * (int64_t)E)) * E;
  auto run = small <= kSmallTiles ? launch_tiles<GATE_UP, 4> : launch_tiles<GATE_UP, 8>;
  return run(A, Wq, Ws, Wz, bias, cnt, off, rows, T, K, N, E, k, G, out, stream);
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
