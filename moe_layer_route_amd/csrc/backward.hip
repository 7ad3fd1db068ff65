// The block's backward pass beside its products and column sums: gradients of the
// routing weights and the router's logits, and the sum of a token's input gradients.
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 2 (router -> top-k softmax
// -> experts -> weighted sum).  For token t with picks j, weights w_j = softmax
// of the picked logits:
//   dw_j = o_j . dy = sum over i of h_j d_j + bd[e_j] . dy    (o_j = h_j . Wd + bd)
//   dl_j = w_j (dw_j - sum over i of w_i dw_i)
//   dx   = sum over j of dxs_j + dl_j Wr[e_j]
// All sums are float32 in a fixed order; the gradients are rounded once to bf16.
// Both are bound by bytes: 16384 slots of H = 2880, dl 25 us (a wave a token, each
// reads dy once and four rows of bd), dx 43 us, 5 TB/s.
#include "device_common.h"
#include "launch.h"

namespace moe {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// ---------------------------------------------------------------------------
// dw and dl: one wave per token; lanes split the columns of dy and bd, and the
// parts of the sums over i that the products left.
// ---------------------------------------------------------------------------
constexpr int kDlWaves = 4;

__global__ __launch_bounds__(kDlWaves * kWave) void backward_dl_kernel(
    const bf16_t* __restrict__ dy, const bf16_t* __restrict__ bd, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ pos, const float* __restrict__ w, const float* __restrict__ dw_part, int parts,
    int64_t T, int H, int k, float* __restrict__ dl) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t t = (int64_t)blockIdx.x * kDlWaves + threadIdx.x / kWave;
  if (t >= T) return;   // wave-uniform, no barrier in this kernel
  const int64_t S = T * k;
  float dw[MOE_MAX_K_DEV];
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j) {
    dw[j] = 0.f;
    if (j < k) {
      const int64_t s = t * k + j;
      const int at = pos[s];
      if (at >= 0) {   // wave-uniform
        float sum = 0.f;
        const u32x4_t* a = reinterpret_cast<const u32x4_t*>(dy + t * H);
        const u32x4_t* b = reinterpret_cast<const u32x4_t*>(bd + (size_t)ids[s] * H);
        for (int c = lane; c < H / 8; c += kWave) {
          const u32x4_t u = a[c], v = b[c];
#pragma unroll
          for (int q = 0; q < 4; ++q) sum = fmaf(bf16hi(u[q]), bf16hi(v[q]), fmaf(bf16lo(u[q]), bf16lo(v[q]), sum));
        }
        for (int q = lane; q < parts; q += kWave) sum += dw_part[(size_t)q * S + at];
        dw[j] = wave_sum(sum);
      }
    }
  }
  float mean = 0.f;
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j)
    if (j < k) mean = fmaf(w[t * k + j], dw[j], mean);
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j)
    if (j < k && lane == j) dl[t * k + j] = w[t * k + j] * (dw[j] - mean);
}

// ---------------------------------------------------------------------------
// dx: one thread per four columns of a token.
// ---------------------------------------------------------------------------
constexpr int kDxThreads = 256;

template <int KMAX>
__global__ __launch_bounds__(kDxThreads) void backward_dx_kernel(const float* __restrict__ dxs,
                                                                 const int32_t* __restrict__ ids,
                                                                 const int32_t* __restrict__ pos,
                                                                 const float* __restrict__ dl,
                                                                 const bf16_t* __restrict__ Wr, int64_t T, int H, int k,
                                                                 bf16_t* __restrict__ dx) {
  const int64_t item = (int64_t)blockIdx.x * kDxThreads + threadIdx.x;
  const int quads = H / 4;
  if (item >= T * quads) return;   // no barrier in this kernel
  const int64_t t = item / quads;
  const int n = 4 * (int)(item - t * quads);
  f32x4_t v[KMAX];
  u32x2_t r[KMAX];
  float f[KMAX];
  bool use[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const size_t s = (size_t)t * k + (j < k ? j : 0);
    const int at = pos[s];
    use[j] = j < k && at >= 0;
    v[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(dxs + (size_t)max(at, 0) * H + n));
    r[j] = *reinterpret_cast<const u32x2_t*>(Wr + (size_t)(at >= 0 ? ids[s] : 0) * H + n);
    f[j] = dl[s];
  }
  f32x4_t a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (use[j]) {
      a[0] += fmaf(f[j], bf16lo(r[j].x), v[j][0]);
      a[1] += fmaf(f[j], bf16hi(r[j].x), v[j][1]);
      a[2] += fmaf(f[j], bf16lo(r[j].y), v[j][2]);
      a[3] += fmaf(f[j], bf16hi(r[j].y), v[j][3]);
    }
  }
  *reinterpret_cast<u32x2_t*>(dx + (size_t)t * H + n) = u32x2_t{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
}

}  // namespace

hipError_t launch_backward_dl(const void* dy, const void* bd, const int32_t* ids, const int32_t* pos, const float* w,
                              const float* dw_part, int parts, int64_t T, int H, int k, float* dl,
                              hipStream_t stream) {
  hipLaunchKernelGGL(backward_dl_kernel, dim3((unsigned)((T + kDlWaves - 1) / kDlWaves)), dim3(kDlWaves * kWave), 0,
                     stream, (const bf16_t*)dy, (const bf16_t*)bd, ids, pos, w, dw_part, parts, T, H, k, dl);
  return hipGetLastError();
}

hipError_t launch_backward_dx_sum(const float* dxs, const int32_t* ids, const int32_t* pos, const float* dl,
                                  const void* Wr, int64_t T, int H, int k, void* dx, hipStream_t stream) {
  const int64_t items = T * (H / 4);
  const dim3 grid((unsigned)((items + kDxThreads - 1) / kDxThreads));
  auto kern = k <= 4 ? backward_dx_kernel<4> : backward_dx_kernel<MOE_MAX_K_DEV>;
  hipLaunchKernelGGL(kern, grid, dim3(kDxThreads), 0, stream, dxs, ids, pos, dl, (const bf16_t*)Wr, T, H, k,
                     (bf16_t*)dx);
  return hipGetLastError();
}

}  // namespace moe
