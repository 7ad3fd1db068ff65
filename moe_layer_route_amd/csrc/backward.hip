// The block's backward pass behind its products: the sum of a token's input
// gradients, and the router's gradients.
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 2 (router -> top-k softmax
// -> experts -> weighted sum).  For token t with picks j, weights w_j = softmax
// of the picked logits:
//   dw_j = o_j . dy = sum over i of h_j d_j + bd[e_j] . dy    (o_j = h_j . Wd + bd)
//   dl_j = w_j (dw_j - sum over i of w_i dw_i)
//   dx   = sum over j of dxs_j + dl_j Wr[e_j]
// All sums are float32 in a fixed order; the gradients are rounded once to bf16.
// (dw and dl are made beside the products.)  Bound by bytes: 16384 slots of H = 2880
// in 50 us, 5 TB/s; a launch of its own for the router took 24 more.
#include "backward_device.h"
#include "launch.h"

namespace moe {
namespace {

#define LDS3 __attribute__((address_space(3)))

// ---------------------------------------------------------------------------
// The first workgroups sum the router's columns (dWr, dbr), the others dx: one
// thread per four columns of a token.
// ---------------------------------------------------------------------------
constexpr int kDxThreads = kSumWaves * kWave;

template <int KMAX>
__global__ __launch_bounds__(kDxThreads) void backward_dx_kernel(
    const float* __restrict__ dxs, const int32_t* __restrict__ ids, const int32_t* __restrict__ pos,
    const float* __restrict__ dl, const bf16_t* __restrict__ Wr, int64_t T, int H, int k, bf16_t* __restrict__ dx,
    const Sum router, const Permuted slots, int sums) {
  __shared__ char smem[kSumLds];
  if ((int)blockIdx.x < sums) {   // workgroup-uniform
    const int e = blockIdx.x / router.parts;
    column_sum<true>(router, slots, e, blockIdx.x - e * router.parts, (LDS3 char*)smem);
    return;
  }
  const int64_t item = (int64_t)(blockIdx.x - sums) * kDxThreads + threadIdx.x;
  const int quads = H / 4;
  if (item >= T * quads) return;   // no barrier from here on
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

hipError_t launch_backward_dx_sum(const float* dxs, const void* x, const int32_t* ids, const int32_t* cnt,
                                  const int32_t* off, const int32_t* rows, const int32_t* pos, const float* dl,
                                  const void* Wr, int64_t T, int H, int E, int k, void* dx, void* dWr, void* dbr,
                                  hipStream_t stream) {
  const Sum router = sum_of(x, dl, H, dWr, dbr);
  const int64_t sums = (int64_t)E * router.parts, blocks = sums + (T * (H / 4) + kDxThreads - 1) / kDxThreads;
  auto kern = k <= 4 ? backward_dx_kernel<4> : backward_dx_kernel<MOE_MAX_K_DEV>;
  hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kDxThreads), 0, stream, dxs, ids, pos, dl, (const bf16_t*)Wr, T,
                     H, k, (bf16_t*)dx, router, Permuted{cnt, off, rows, per_token(k)}, (int)sums);
  return hipGetLastError();
}

}  // namespace moe
