// MXFP4 rows: bf16 rows to E2M1 codes with one power of two per 32 values, and
// back (the activations of the products with 4 bits on both sides).
//
// xserv "Phase 19: gpt-oss-20b MoE support", section 5 (MXFP4).  Codes uint8
// [R][K/2], the even k in the low half of a byte; scales uint8
// [ceil(K/128)][R][4]: the four blocks of 128 values of a row are one word, and
// the words of neighbouring rows lie side by side, as the products load them.
//
// Bound by bytes: 2 K + K/2 + K/32 a row in either direction.  A row of 16
// lanes takes 128 values of a row, so a quad of lanes has one block (16 bytes a
// lane, its maximum two lane moves away) and the row of lanes one scale word;
// a wave's loads are four 256-byte runs and its four scale words one 16-byte
// run.  Both directions over 16384 rows of 2880: 51.5 us, 4.6 TB/s, 94% of a plain
// copy's rate; over one row 10.9 us, of which the two launches are nearly all.
#include "launch.h"
#include "mxfp4_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerWg = kThreads / 16;

__global__ __launch_bounds__(kThreads) void mxfp4_rows_kernel(const bf16_t* __restrict__ a, int64_t r_begin,
                                                             int64_t R, int K, uint32_t* __restrict__ codes,
                                                             uint32_t* __restrict__ scales) {
  const int64_t r = r_begin + (int64_t)blockIdx.x * kRowsPerWg + threadIdx.x / 16;
  quantize_128(a, r, R, K, blockIdx.y, threadIdx.x % 16, codes, scales);
}

__global__ __launch_bounds__(kThreads) void mxfp4_rows_back_kernel(const uint32_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  int64_t r_begin, int64_t R, int K,
                                                                  bf16_t* __restrict__ out) {
  const int64_t r = r_begin + (int64_t)blockIdx.x * kRowsPerWg + threadIdx.x / 16;
  const int l = threadIdx.x % 16, group = blockIdx.y;
  const int k = 128 * group + 8 * l;
  if (r >= R || k >= K) return;   // no barrier in this kernel
  const uint32_t c = codes[(r * K + k) / 8];
  const uint32_t s = scales[((int64_t)group * R + r) * 4 + l / 4];
  *reinterpret_cast<u32x4_t*>(out + r * K + k) = dequant8(c, ue8m0_to_f32(s));
}

// A launch takes at most 2^27 rows (its grid has fewer than 2^32 threads along x).
template <class F>
hipError_t in_parts(int64_t R, int K, F launch) {
  constexpr int64_t kPart = (int64_t)1 << 27;
  for (int64_t r0 = 0; r0 < R; r0 += kPart) {
    const int64_t n = R - r0 < kPart ? R - r0 : kPart;
    launch(r0, dim3((unsigned)((n + kRowsPerWg - 1) / kRowsPerWg), (unsigned)((K + 127) / 128)));
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mxfp4_rows(const void* a, int64_t R, int K, void* codes, void* scales, hipStream_t stream) {
  return in_parts(R, K, [&](int64_t r0, dim3 grid) {
    hipLaunchKernelGGL(mxfp4_rows_kernel, grid, dim3(kThreads), 0, stream, (const bf16_t*)a, r0, R, K,
                       (uint32_t*)codes, (uint32_t*)scales);
  });
}

hipError_t launch_mxfp4_rows_back(const void* codes, const void* scales, int64_t R, int K, void* out,
                                  hipStream_t stream) {
  return in_parts(R, K, [&](int64_t r0, dim3 grid) {
    hipLaunchKernelGGL(mxfp4_rows_back_kernel, grid, dim3(kThreads), 0, stream, (const uint32_t*)codes,
                       (const uint8_t*)scales, r0, R, K, (bf16_t*)out);
  });
}

}  // namespace moe
