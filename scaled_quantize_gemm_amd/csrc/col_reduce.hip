#include "col_reduce.h"

namespace sfp8 {

// 64 columns per block (a column per lane), the partial rows over 4 waves, joined in LDS
__global__ void __launch_bounds__(256) col_reduce_kernel(const float* __restrict__ part, int parts, int64_t n,
                                                         float* __restrict__ out, int64_t split, float* __restrict__ out2) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < n)
    for (int p = wave; p < parts; p += 4) s += part[p * n + c];
  red[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= n) return;
  s = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
  if (c < split) out[c] = s;
  else if (out2 != nullptr) out2[c - split] = s;
}

void launch_col_reduce(const float* part, int parts, int64_t n, float* out, int64_t split, float* out2, hipStream_t st) {
  hipLaunchKernelGGL(col_reduce_kernel, dim3((unsigned)((n + 63) / 64)), dim3(256), 0, st, part, parts, n, out, split,
                     out2);
}

}  // namespace sfp8
