#include "col_reduce.h"

namespace sfp8 {

// 64 columns per block (a column per lane), a segment per grid row, the partial rows over 16 waves, each wave's loads 8 in
// flight; joined in LDS
constexpr int kCrWaves = 16;
__global__ void __launch_bounds__(64 * kCrWaves) col_reduce_kernel(const float* __restrict__ part, int parts, int segs,
                                                                   int64_t pitch, int64_t n, float* __restrict__ out,
                                                                   float* __restrict__ out2) {
  __shared__ float red[kCrWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane, stride = segs * pitch;
  const float* src = part + blockIdx.y * pitch + c;
  float s = 0.0f;
  if (c < n) {
    int p = wave;
    for (; p + 7 * kCrWaves < parts; p += 8 * kCrWaves) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = src[(p + k * kCrWaves) * stride];
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; p < parts; p += kCrWaves) s += src[p * stride];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= n) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < kCrWaves; ++k) s += red[k][lane];
  (blockIdx.y == 0 ? out : out2)[c] = s;
}

void launch_col_reduce(const float* part, int parts, int segs, int64_t pitch, int64_t n, float* out, float* out2,
                       hipStream_t st) {
  hipLaunchKernelGGL(col_reduce_kernel, dim3((unsigned)((n + 63) / 64), out2 != nullptr ? 2 : 1), dim3(64 * kCrWaves), 0,
                     st, part, parts, segs, pitch, n, out, out2);
}

}  // namespace sfp8
