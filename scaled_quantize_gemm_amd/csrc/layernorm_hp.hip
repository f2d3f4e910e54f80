// LayerNorm with a high-precision output, and its backward pass.
//
//   mean = sum(x) / cols, var = sum((x - mean)^2) / cols, rs = 1 / sqrt(var + eps)
//   y = (x - mean) rs gamma + beta
//   dx = rs (g - mean(g) - xh mean(g xh)) + dres,  g = dy gamma,  xh = (x - mean) rs
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy
// One wave per row, the row read once per pass; dgamma and dbeta over chunks of rows, then joined.
#include <algorithm>

#include "col_reduce.h"

namespace sfp8 {

constexpr int64_t kLnMaxCols = 32768;

template <bool BF16>
__device__ __forceinline__ float ln_ld(const void* __restrict__ p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ float ln_ldw(const void* __restrict__ p, int bf16, int64_t i) {
  return bf16 ? ln_ld<true>(p, i) : ln_ld<false>(p, i);
}
template <bool BF16>
__device__ __forceinline__ void ln_st(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_bits(v);
  else static_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ float ln_wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <bool XBF, bool YBF>
__global__ void __launch_bounds__(256) ln_fwd_kernel(const void* x, const void* __restrict__ gamma,
                                                     const void* __restrict__ beta, int w_bf16, float eps, int64_t rows,
                                                     int cols, void* y, float* __restrict__ mu, float* __restrict__ rs_out) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t base = row * cols;
  float s = 0.0f;
  for (int c = lane; c < cols; c += 64) s += ln_ld<XBF>(x, base + c);
  const float mean = ln_wave_sum(s) / (float)cols;
  float q = 0.0f;
  for (int c = lane; c < cols; c += 64) {
    const float d = ln_ld<XBF>(x, base + c) - mean;
    q += d * d;
  }
  const float rs = 1.0f / sqrtf(ln_wave_sum(q) / (float)cols + eps);
  if (lane == 0) {
    if (mu != nullptr) mu[row] = mean;
    if (rs_out != nullptr) rs_out[row] = rs;
  }
  for (int c = lane; c < cols; c += 64) {
    const float v = (ln_ld<XBF>(x, base + c) - mean) * rs;
    const float g = ln_ldw(gamma, w_bf16, c);
    ln_st<YBF>(y, base + c, beta != nullptr ? fmaf(v, g, ln_ldw(beta, w_bf16, c)) : v * g);
  }
}

// dgamma and dbeta of a chunk of rows: a column per lane, the chunk's rows over 4 waves
constexpr int kLnChunk = 128;
template <bool XBF, bool DBF>
__global__ void __launch_bounds__(256) ln_wgrad_kernel(const void* __restrict__ dy, const void* __restrict__ x,
                                                       const float* __restrict__ mu, const float* __restrict__ rsig,
                                                       int64_t rows, int cols, float* __restrict__ part) {
  __shared__ float red[2][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.y * 64 + lane;
  const int64_t r0 = (int64_t)blockIdx.x * kLnChunk, r1 = r0 + kLnChunk < rows ? r0 + kLnChunk : rows;
  float dg = 0.0f, db = 0.0f;
  if (c < cols)
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      const float d = ln_ld<DBF>(dy, r * cols + c);
      dg += d * ((ln_ld<XBF>(x, r * cols + c) - mu[r]) * rsig[r]);
      db += d;
    }
  red[0][wave][lane] = dg;
  red[1][wave][lane] = db;
  __syncthreads();
  if (wave < 2 && c < cols) {
    const float* v = red[wave][0] + lane;
    part[((int64_t)blockIdx.x * 2 + wave) * cols + c] = (v[0] + v[64]) + (v[128] + v[192]);
  }
}

template <bool XBF, bool DBF>
__global__ void __launch_bounds__(256) ln_dx_kernel(const void* dy, const void* __restrict__ x,
                                                    const void* __restrict__ gamma, int w_bf16,
                                                    const float* __restrict__ mu, const float* __restrict__ rsig,
                                                    const void* dres, int64_t rows, int cols, void* dx) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int64_t base = row * cols;
  const float m = mu[row], rs = rsig[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int c = lane; c < cols; c += 64) {
    const float g = ln_ld<DBF>(dy, base + c) * ln_ldw(gamma, w_bf16, c);
    s1 += g;
    s2 += g * ((ln_ld<XBF>(x, base + c) - m) * rs);
  }
  s1 = ln_wave_sum(s1) / (float)cols;
  s2 = ln_wave_sum(s2) / (float)cols;
  for (int c = lane; c < cols; c += 64) {
    const float g = ln_ld<DBF>(dy, base + c) * ln_ldw(gamma, w_bf16, c);
    float d = rs * (g - s1 - (ln_ld<XBF>(x, base + c) - m) * rs * s2);
    if (dres != nullptr) d += ln_ld<XBF>(dres, base + c);
    ln_st<XBF>(dx, base + c, d);
  }
}

}  // namespace sfp8

using namespace sfp8;

extern "C" int fp8_layernorm(const void* x, int x_dtype, int64_t rows, int64_t cols, const void* gamma,
                             const void* beta, int w_dtype, float eps, void* y, int y_dtype, float* mu, float* rsigma,
                             void* stream) {
  const char* what = "fp8_layernorm";
  SFP8_REQUIRE(x_dtype == HP_F32 || x_dtype == HP_BF16, FP8_ERR_DTYPE, "%s: x_dtype %d", what, x_dtype);
  SFP8_REQUIRE(w_dtype == HP_F32 || w_dtype == HP_BF16, FP8_ERR_DTYPE, "%s: w_dtype %d", what, w_dtype);
  SFP8_REQUIRE(y_dtype == OUT_F32 || y_dtype == OUT_BF16, FP8_ERR_DTYPE, "%s: y_dtype %d", what, y_dtype);
  SFP8_REQUIRE(rows >= 0 && cols >= 0, FP8_ERR_SHAPE, "%s: negative shape", what);
  SFP8_REQUIRE(rows < (1ll << 31) && cols <= kLnMaxCols, FP8_ERR_SHAPE, "%s: rows=%lld (< 2^31) cols=%lld (<= %lld)",
               what, (long long)rows, (long long)cols, (long long)kLnMaxCols);
  SFP8_REQUIRE(eps >= 0.0f, FP8_ERR_ARG, "%s: eps must be >= 0", what);
  if (rows == 0 || cols == 0) return FP8_OK;
  SFP8_REQUIRE(x != nullptr && y != nullptr && gamma != nullptr, FP8_ERR_ARG, "%s: null x, y or gamma", what);
  SFP8_REQUIRE(aligned16(x) && aligned16(y) && aligned16(gamma) && aligned16(beta), FP8_ERR_ARG,
               "%s: x, y, gamma, beta must be 16-byte aligned", what);
  SFP8_REQUIRE(aligned4(mu) && aligned4(rsigma), FP8_ERR_ARG, "%s: misaligned mu / rsigma", what);
  SFP8_REQUIRE(x != y || (x_dtype == HP_BF16) == (y_dtype == OUT_BF16), FP8_ERR_ARG,
               "%s: y may be x only where both have one type", what);
  hipStream_t st = (hipStream_t)stream;
  const dim3 grid((unsigned)((rows + 3) / 4));
  const int wb = w_dtype == HP_BF16, c = (int)cols;
#define SFP8_LN_FWD(X, Y) \
  hipLaunchKernelGGL((ln_fwd_kernel<X, Y>), grid, dim3(256), 0, st, x, gamma, beta, wb, eps, rows, c, y, mu, rsigma)
  if (x_dtype == HP_BF16) {
    if (y_dtype == OUT_BF16) SFP8_LN_FWD(true, true);
    else SFP8_LN_FWD(true, false);
  } else {
    if (y_dtype == OUT_BF16) SFP8_LN_FWD(false, true);
    else SFP8_LN_FWD(false, false);
  }
#undef SFP8_LN_FWD
  return check_launch(what);
}

extern "C" size_t fp8_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= (1ll << 31) || cols < 0 || cols > kLnMaxCols) return 0;
  return (size_t)((rows + kLnChunk - 1) / kLnChunk) * 2 * (size_t)cols * sizeof(float);
}

extern "C" int fp8_layernorm_backward(const void* dy, int dy_dtype, const void* x, int x_dtype, int64_t rows,
                                      int64_t cols, const void* gamma, int w_dtype, const float* mu,
                                      const float* rsigma, const void* dres, void* dx, float* dgamma, float* dbeta,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* what = "fp8_layernorm_backward";
  SFP8_REQUIRE(dy_dtype == HP_F32 || dy_dtype == HP_BF16, FP8_ERR_DTYPE, "%s: dy_dtype %d", what, dy_dtype);
  SFP8_REQUIRE(x_dtype == HP_F32 || x_dtype == HP_BF16, FP8_ERR_DTYPE, "%s: x_dtype %d", what, x_dtype);
  SFP8_REQUIRE(w_dtype == HP_F32 || w_dtype == HP_BF16, FP8_ERR_DTYPE, "%s: w_dtype %d", what, w_dtype);
  SFP8_REQUIRE(rows >= 0 && cols >= 0, FP8_ERR_SHAPE, "%s: negative shape", what);
  SFP8_REQUIRE(rows < (1ll << 31) && cols <= kLnMaxCols, FP8_ERR_SHAPE, "%s: rows=%lld (< 2^31) cols=%lld (<= %lld)",
               what, (long long)rows, (long long)cols, (long long)kLnMaxCols);
  if (cols == 0) return FP8_OK;
  SFP8_REQUIRE(dgamma != nullptr && aligned4(dgamma) && aligned4(dbeta), FP8_ERR_ARG,
               "%s: dgamma must be non-null, dgamma and dbeta 4-byte aligned", what);
  hipStream_t st = (hipStream_t)stream;
  const int wb = w_dtype == HP_BF16, c = (int)cols;
  const int64_t chunks = (rows + kLnChunk - 1) / kLnChunk;
  float* part = static_cast<float*>(workspace);
  if (rows > 0) {
    SFP8_REQUIRE(dy != nullptr && x != nullptr && gamma != nullptr && mu != nullptr && rsigma != nullptr && dx != nullptr,
                 FP8_ERR_ARG, "%s: null dy, x, gamma, mu, rsigma or dx", what);
    SFP8_REQUIRE(aligned16(dy) && aligned16(x) && aligned16(gamma) && aligned16(dres) && aligned16(dx), FP8_ERR_ARG,
                 "%s: dy, x, gamma, dres, dx must be 16-byte aligned", what);
    SFP8_REQUIRE(aligned4(mu) && aligned4(rsigma), FP8_ERR_ARG, "%s: misaligned mu / rsigma", what);
    SFP8_REQUIRE(dx != dy || dy_dtype == x_dtype, FP8_ERR_ARG, "%s: dx may be dy only where dy has x's type", what);
    SFP8_REQUIRE(dx != x, FP8_ERR_ARG, "%s: dx may not be x", what);
    const size_t need = fp8_layernorm_backward_workspace(rows, cols);
    SFP8_REQUIRE(workspace != nullptr && aligned16(workspace) && workspace_bytes >= need, FP8_ERR_ARG,
                 "%s: workspace of %zu bytes, 16-byte aligned, needed (%zu given)", what, need, workspace_bytes);
    const dim3 wgrid((unsigned)chunks, (unsigned)((cols + 63) / 64)), grid((unsigned)((rows + 3) / 4));
#define SFP8_LN_BWD(X, D)                                                                                          \
  do {                                                                                                             \
    hipLaunchKernelGGL((ln_wgrad_kernel<X, D>), wgrid, dim3(256), 0, st, dy, x, mu, rsigma, rows, c, part);        \
    hipLaunchKernelGGL((ln_dx_kernel<X, D>), grid, dim3(256), 0, st, dy, x, gamma, wb, mu, rsigma, dres, rows, c,  \
                       dx);                                                                                        \
  } while (0)
    if (x_dtype == HP_BF16) {
      if (dy_dtype == HP_BF16) SFP8_LN_BWD(true, true);
      else SFP8_LN_BWD(true, false);
    } else {
      if (dy_dtype == HP_BF16) SFP8_LN_BWD(false, true);
      else SFP8_LN_BWD(false, false);
    }
#undef SFP8_LN_BWD
    const int rc = check_launch(what);
    if (rc != FP8_OK) return rc;
  }
  launch_col_reduce(part, (int)chunks, 2 * cols, dgamma, cols, dbeta, st);
  return check_launch(what);
}
