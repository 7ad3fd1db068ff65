// Router and permutation of a call with few token slots, in two launches.
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 2 (router, top-k, softmax
// over the picks; the ids stay on the GPU).  The decision is the exact
// router's: products of bf16 values and their sums in float64, the order by
// the float32 logit (descending, then the lower index), the softmax in float64.
//
// The exact router gives a token one workgroup, which reads the whole router
// weight through one CU; here the logits are spread over the card first, and
// one workgroup then picks and permutes.
#include "device_common.h"
#include "launch.h"
#include "route_key.h"
#include "wave_reduce.h"

namespace moe {
namespace {

// One workgroup per EB experts x TB tokens; its waves split K.
constexpr int kLogitThreads = 256;

template <int EB, int TB>
__global__ __launch_bounds__(kLogitThreads) void few_logits_kernel(const bf16_t* __restrict__ x,
                                                                   const bf16_t* __restrict__ Wr,
                                                                   const bf16_t* __restrict__ br, int T, int H, int E,
                                                                   double* __restrict__ logits) {
  constexpr int kWaves = kLogitThreads / kWave;
  __shared__ double part[kWaves][EB * TB];
  const int e0 = blockIdx.x * EB, t0 = blockIdx.y * TB;
  const u32x4_t *xr[TB], *wr[EB];
#pragma unroll
  for (int t = 0; t < TB; ++t) xr[t] = reinterpret_cast<const u32x4_t*>(x + (size_t)min(t0 + t, T - 1) * H);
#pragma unroll
  for (int e = 0; e < EB; ++e) wr[e] = reinterpret_cast<const u32x4_t*>(Wr + (size_t)min(e0 + e, E - 1) * H);
  double sum[EB][TB];
#pragma unroll
  for (int e = 0; e < EB; ++e)
#pragma unroll
    for (int t = 0; t < TB; ++t) sum[e][t] = 0.0;
  for (int i = threadIdx.x; i < H / 8; i += kLogitThreads) {
    u32x4_t a[TB], b[EB];
#pragma unroll
    for (int t = 0; t < TB; ++t) a[t] = xr[t][i];
#pragma unroll
    for (int e = 0; e < EB; ++e) b[e] = wr[e][i];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      double bl[EB], bh[EB];
#pragma unroll
      for (int e = 0; e < EB; ++e) bl[e] = (double)bf16lo(b[e][q]), bh[e] = (double)bf16hi(b[e][q]);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const double al = (double)bf16lo(a[t][q]), ah = (double)bf16hi(a[t][q]);
#pragma unroll
        for (int e = 0; e < EB; ++e) sum[e][t] = __builtin_fma(ah, bh[e], __builtin_fma(al, bl[e], sum[e][t]));
      }
    }
  }
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int e = 0; e < EB; ++e)
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const double s = wave_add(sum[e][t]);
      if (lane == 0) part[wave][e * TB + t] = s;
    }
  __syncthreads();
  const int e = e0 + (int)threadIdx.x / TB, t = t0 + (int)threadIdx.x % TB;
  if (threadIdx.x < EB * TB && e < E && t < T) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += part[w][threadIdx.x];
    logits[(size_t)t * E + e] = s + (double)bf16_to_f32(br[e]);
  }
}

// The picks, their weights and the stable permutation of the slots of up to 64
// tokens, by one workgroup.  Sixteen lanes take a token, four tokens a wave:
// lane c holds experts c, c + 16, ... (16 KEYS of them), and a reduction stays
// within a row of lanes.  Then thread s takes slot s (k <= 8: there are fewer
// slots than threads), as in the permutation's own kernel: equal ids of a wave by
// ballots over the id's bits, counts per wave and expert, and their sums in the
// order of the waves.
constexpr int kMaxTokens = 64;
constexpr int kMaxThreads = 16 * kMaxTokens;
constexpr int kSlotWaves = kMaxTokens * MOE_MAX_K_DEV / kWave;

template <int KEYS>
__global__ __launch_bounds__(kMaxThreads) void few_decide_kernel(
    const double* __restrict__ logits, int T, int E, int k, const int32_t* __restrict__ n_valid, int e_begin,
    int n_local, int32_t* __restrict__ ids, float* __restrict__ w, int32_t* __restrict__ cnt,
    int32_t* __restrict__ off, int32_t* __restrict__ rows, int32_t* __restrict__ pos) {
  __shared__ int count[kSlotWaves][MOE_MAX_E_DEV];   // per wave and expert, then what precedes it
  __shared__ int first[MOE_MAX_E_DEV];               // an expert's count, then its first row
  __shared__ int slot_id[kMaxThreads];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int i = tid; i < kSlotWaves * MOE_MAX_E_DEV; i += blockDim.x) (&count[0][0])[i] = 0;
  slot_id[tid] = -1;
  __syncthreads();

  const int valid = n_valid ? *n_valid : T;
  const int c = lane & 15, row = lane & ~15;
  const int t = tid / 16;
  const double* l = logits + (size_t)min(t, T - 1) * E;
  uint64_t key[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; ++i) key[i] = c + 16 * i < E ? make_key((float)l[c + 16 * i], c + 16 * i) : 0;
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < KEYS; ++i) best = key[i] > best ? key[i] : best;
    const int e = key_expert(row_max(best));
#pragma unroll
    for (int i = 0; i < KEYS; ++i) key[i] = c + 16 * i == e ? 0 : key[i];
    if (c == j) mine = e;
  }
  const double lm = l[mine], top = __shfl(lm, row), z = c < k ? exp(lm - top) : 0.0;
  double sum = 0.0;
  for (int j = 0; j < k; ++j) sum += __shfl(z, row + j);
  if (c < k && t < T) {
    const bool real = t < valid;
    ids[t * k + c] = real ? mine : -1;
    w[t * k + c] = real ? (float)(z / sum) : 0.0f;
    const int e = mine - e_begin;
    if (real && (unsigned)e < (unsigned)n_local) slot_id[t * k + c] = e;
  }
  __syncthreads();

  const int e = slot_id[tid];
  uint64_t peers = __ballot(e >= 0);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool bit = (e >> b) & 1;
    const uint64_t with = __ballot(bit);
    peers &= bit ? with : ~with;
  }
  const int rank = __popcll(peers & ((1ull << lane) - 1));
  if (e >= 0 && rank == 0) count[wave][e] = __popcll(peers);
  __syncthreads();
  for (int i = tid; i < n_local; i += blockDim.x) {
    int n[kSlotWaves], run = 0;
#pragma unroll
    for (int v = 0; v < kSlotWaves; ++v) n[v] = count[v][i];
#pragma unroll
    for (int v = 0; v < kSlotWaves; ++v) {
      count[v][i] = run;
      run += n[v];
    }
    first[i] = run;
  }
  __syncthreads();
  if (wave == 0) {
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = lane * 4 + i < n_local ? first[lane * 4 + i] : 0;
      sum += n[i];
    }
    const int incl = wave_incl_scan(sum, lane);
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = lane * 4 + i;
      if (at < n_local) {
        cnt[at] = n[i];
        off[at] = run;
        first[at] = run;
      }
      run += n[i];
    }
    if (lane == kWave - 1) off[n_local] = incl;
  }
  __syncthreads();
  if (tid < T * k) {
    const int p = e < 0 ? -1 : first[e] + count[wave][e] + rank;
    pos[tid] = p;
    if (e >= 0) rows[p] = tid;
  }
}

}  // namespace

hipError_t launch_few_logits(const void* x, const void* Wr, const void* br, int64_t T, int H, int E, double* logits,
                             hipStream_t stream) {
  const bool blocks = T >= 4;
  const int eb = blocks ? 2 : 1, tb = blocks ? 4 : 1;
  auto kern = blocks ? few_logits_kernel<2, 4> : few_logits_kernel<1, 1>;
  hipLaunchKernelGGL(kern, dim3((unsigned)((E + eb - 1) / eb), (unsigned)((T + tb - 1) / tb)), dim3(kLogitThreads), 0,
                     stream, (const bf16_t*)x, (const bf16_t*)Wr, (const bf16_t*)br, (int)T, H, E, logits);
  return hipGetLastError();
}

// One round of tokens, and o of T k x H floats must hold T x E doubles.  (Block
// of int4 experts, against the exact router and the permutation: 8 tokens of 32
// experts 60.0 against 64.6 us, 16 of 128 123 against 137, 64 of 32 87.9 against
// 90.3; with further rounds 128 of 32 113.3 against 112.7, 256 of 32 198 against
// 193.)
bool takes_few(int64_t T, int H, int E, int k) { return T <= kMaxTokens && (int64_t)k * H >= 2 * (int64_t)E; }

hipError_t launch_few_route(const void* x, const void* Wr, const void* br, int64_t T, int H, int E, int k,
                            const int32_t* n_valid, int e_begin, int n_local, double* logits, int32_t* ids, float* w,
                            int32_t* cnt, int32_t* off, int32_t* rows, int32_t* pos, hipStream_t stream) {
  if (T > kMaxTokens) return hipErrorInvalidValue;
  hipError_t err = launch_few_logits(x, Wr, br, T, H, E, logits, stream);
  if (err != hipSuccess) return err;
  const int waves = (int)(T + 3) / 4;
  hipLaunchKernelGGL(E <= 64 ? few_decide_kernel<4> : few_decide_kernel<16>, dim3(1), dim3(waves * kWave), 0, stream,
                     logits, (int)T, E, k, n_valid, e_begin, n_local, ids, w, cnt, off, rows, pos);
  return hipGetLastError();
}

}  // namespace moe
