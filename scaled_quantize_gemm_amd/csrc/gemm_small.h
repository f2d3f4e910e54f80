// FP8 x FP8 GEMM kernels on gfx950 matrix cores: C[M][N] = sum_k deq(A[m][k]) deq(B[n][k]),
// templated on the epilogue (gemm_epilogue.h) so that the plain and the fused entry points
// (gemm.hip, gemm_fused.hip) share them.
//
// "Week 14" course page: matmuls run in FP8 (FP8 bullet); FP8 products are summed in a
// wider accumulator and partial sums promoted to fp32 at fixed intervals
// (accumulation-precision bullet); MX gives every 32 numbers a shared scale and DeepSeek-V3
// scales 1x128 activation runs and 128x128 weight blocks (absmax bullet).
//
// Matrix-core facts this kernel is built on (gfx950, v_mfma_*_16x16x128_f8f6f4):
//  * operand layout: lane l = 16 g + r supplies row r of its 16-row operand; its 32 bytes are
//    K = 16g .. 16g+15 (bytes 0-15) and K = 64+16g .. 64+16g+15 (bytes 16-31);
//  * result layout: lane l holds C[4g + j][r], j = 0..3;
//  * scaled form: lane l's e8m0 byte scales row r over K = 32g .. 32g+31 by 2^(e - 127);
//  * the products are exact; runs of 8 consecutive K are summed in a fixed-point window
//    below the run's largest product, and each run is promoted into the fp32 accumulator.
//
// Block tile BM x BN x 128, 4 waves in a 2 x 2 grid, each wave (BM/2) x (BN/2) built from
// 16x16x128 MFMAs.  A and B tiles are staged through LDS (double-buffered, 16-byte chunks
// XOR-swizzled by row so the fragment reads of 16 consecutive rows hit distinct banks).
//
// Scaling modes:
//  * TENSOR:  acc over all K; C = acc * (sa * sb).
//  * BLOCK:   per 128-K block kb: p = MFMA from zero; acc += p * (sa[kb][m] * sb[n/128][kb]).
//  * TILE2:   both operands in 1x128 runs along K: acc += p * (sa[kb][m] * sb[kb][n]).
//  * MX:      scaled MFMA with the e8m0 codes of A[m][4kb+g] and B[n][4kb+g]; C = acc.
#pragma once

#include "gemm_common.h"

namespace sfp8 {

template <int BM, int BN>
struct GemmCfg {
  static constexpr int BK = 128;
  static constexpr int WM = BM / 2, WN = BN / 2;  // wave tile
  static constexpr int TM = WM / 16, TN = WN / 16;  // MFMA tiles per wave
  static constexpr int A_CHUNKS = BM * BK / 16, B_CHUNKS = BN * BK / 16;
  static constexpr int A_PER_T = A_CHUNKS / 256, B_PER_T = B_CHUNKS / 256;
  static constexpr int LDS_A = BM * BK, LDS_B = BN * BK;  // bytes per stage
};

// byte offset of 16-byte chunk c of tile row `row` in a 128-byte-row LDS tile; the position
// c ^ ((row >> 1) ^ ((row & 1) << 2)) is distinct over any 8 consecutive rows (32 banks) and
// over 16 consecutive rows for each row parity (64 banks), so fragment reads do not conflict
__device__ __forceinline__ int swz(int row, int c) { return row * 128 + ((c ^ (((row >> 1) ^ ((row & 1) << 2)) & 7)) << 4); }

template <int BM, int BN, int MODE, int FA, int FB, int OUT, int EPI>
__global__ void __launch_bounds__(256) gemm_kernel(const uint8_t* __restrict__ A, const uint8_t* __restrict__ B,
                                                   const void* __restrict__ sa_p, const void* __restrict__ sb_p,
                                                   const EpiParams ep, int M, int N, int K) {
  using Cfg = GemmCfg<BM, BN>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint8_t* lds_a = smem;                      // [2][BM][128]
  uint8_t* lds_b = smem + 2 * Cfg::LDS_A;     // [2][BN][128]

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int g = lane >> 4, r = lane & 15;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
  const int nk = K / 128;

  // ---- global -> register staging of one K-step
  uint4 ra[Cfg::A_PER_T], rb[Cfg::B_PER_T];
  auto load_step = [&](int ks) {
#pragma unroll
    for (int i = 0; i < Cfg::A_PER_T; ++i) {
      const int id = tid + 256 * i, row = id >> 3, c = id & 7;
      int gm = m0 + row;
      gm = gm < M ? gm : M - 1;
      ra[i] = *reinterpret_cast<const uint4*>(A + (size_t)gm * K + (size_t)ks * 128 + c * 16);
    }
#pragma unroll
    for (int i = 0; i < Cfg::B_PER_T; ++i) {
      const int id = tid + 256 * i, row = id >> 3, c = id & 7;
      int gn = n0 + row;
      gn = gn < N ? gn : N - 1;
      rb[i] = *reinterpret_cast<const uint4*>(B + (size_t)gn * K + (size_t)ks * 128 + c * 16);
    }
  };
  auto store_step = [&](int buf) {
#pragma unroll
    for (int i = 0; i < Cfg::A_PER_T; ++i) {
      const int id = tid + 256 * i, row = id >> 3, c = id & 7;
      *reinterpret_cast<uint4*>(lds_a + buf * Cfg::LDS_A + swz(row, c)) = ra[i];
    }
#pragma unroll
    for (int i = 0; i < Cfg::B_PER_T; ++i) {
      const int id = tid + 256 * i, row = id >> 3, c = id & 7;
      *reinterpret_cast<uint4*>(lds_b + buf * Cfg::LDS_B + swz(row, c)) = rb[i];
    }
  };

  v4f acc[Cfg::TM][Cfg::TN];
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  if (nk > 0) {
    load_step(0);
    store_step(0);
  }
  __syncthreads();

  for (int ks = 0; ks < nk; ++ks) {
    const int buf = ks & 1;
    if (ks + 1 < nk) load_step(ks + 1);

    // ---- per-step scale operands
    float sab[Cfg::TM][4], sbc[Cfg::TN];
    int scale_a[Cfg::TM], scale_b[Cfg::TN];
    if constexpr (MODE == MODE_BLOCK || MODE == MODE_TILE2) {
      const float* sa = static_cast<const float*>(sa_p);
      const float* sb = static_cast<const float*>(sb_p);
      const float sbv = MODE == MODE_BLOCK ? sb[(size_t)(n0 / 128) * nk + ks] : 1.0f;
      if constexpr (MODE == MODE_TILE2) {
#pragma unroll
        for (int j = 0; j < Cfg::TN; ++j) {
          int gn = n0 + wn * Cfg::WN + 16 * j + r;
          gn = gn < N ? gn : N - 1;
          sbc[j] = sb[(size_t)ks * N + gn];  // [K/128][N]
        }
      }
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          int gm = m0 + wm * Cfg::WM + 16 * i + 4 * g + j;
          gm = gm < M ? gm : M - 1;
          sab[i][j] = sa[(size_t)ks * M + gm] * sbv;
        }
    }
    if constexpr (MODE == MODE_MX) {
      const uint8_t* ea = static_cast<const uint8_t*>(sa_p);
      const uint8_t* eb = static_cast<const uint8_t*>(sb_p);
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i) {
        int gm = m0 + wm * Cfg::WM + 16 * i + r;
        gm = gm < M ? gm : M - 1;
        scale_a[i] = ea[(size_t)(4 * ks + g) * M + gm];  // e8m0 layout [K/32][M]
      }
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j) {
        int gn = n0 + wn * Cfg::WN + 16 * j + r;
        gn = gn < N ? gn : N - 1;
        scale_b[j] = eb[(size_t)(4 * ks + g) * N + gn];
      }
    }

    // ---- fragments from LDS
    v8i fa[Cfg::TM], fb[Cfg::TN];
#pragma unroll
    for (int i = 0; i < Cfg::TM; ++i) {
      const int row = wm * Cfg::WM + 16 * i + r;
      const uint8_t* base = lds_a + buf * Cfg::LDS_A;
      uint4 lo = *reinterpret_cast<const uint4*>(base + swz(row, g));
      uint4 hi = *reinterpret_cast<const uint4*>(base + swz(row, g + 4));
      fa[i] = v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    }
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j) {
      const int row = wn * Cfg::WN + 16 * j + r;
      const uint8_t* base = lds_b + buf * Cfg::LDS_B;
      uint4 lo = *reinterpret_cast<const uint4*>(base + swz(row, g));
      uint4 hi = *reinterpret_cast<const uint4*>(base + swz(row, g + 4));
      fb[j] = v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    }

    // ---- matrix cores
#pragma unroll
    for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j) {
        if constexpr (MODE == MODE_TENSOR) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[i], fb[j], acc[i][j], FA, FB, 0, 0, 0, 0);
        } else if constexpr (MODE == MODE_MX) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[i], fb[j], acc[i][j], FA, FB, 0, scale_a[i],
                                                                        0, scale_b[j]);
        } else {
          v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[i], fb[j], v4f{0.f, 0.f, 0.f, 0.f}, FA, FB, 0,
                                                                    0, 0, 0);
#pragma unroll
          for (int jj = 0; jj < 4; ++jj)
            acc[i][j][jj] = fmaf(p[jj], MODE == MODE_TILE2 ? sab[i][jj] * sbc[j] : sab[i][jj], acc[i][j][jj]);
        }
      }

    if (ks + 1 < nk) store_step(buf ^ 1);
    __syncthreads();
  }

  // ---- epilogue: lane (g, r) holds column 16j + r of rows 4g + jj of tile (i, j)
  Epilogue<OUT, EPI> epi(ep);
  float s = 1.0f;
  if constexpr (MODE == MODE_TENSOR) s = *static_cast<const float*>(sa_p) * *static_cast<const float*>(sb_p);
  epi.with_act([&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j) {
      const int gn = n0 + wn * Cfg::WN + 16 * j + r;
      float b[1];
      epi.template bias<1>(gn, N, b);
      // the residual of this column's rows (for SwiGLU the gate columns' lanes) before the first store
      constexpr int W = ACT == FP8_ACT_SWIGLU ? 2 : 1;
      typename Epilogue<OUT, EPI>::template Run<ACT, W> res[EPI == EPI_RESIDUAL ? 4 * Cfg::TM : 1];
      if constexpr (EPI == EPI_RESIDUAL) {
#pragma unroll
        for (int k = 0; k < 4 * Cfg::TM; ++k) {
          const int gm = m0 + wm * Cfg::WM + 16 * (k >> 2) + 4 * g + (k & 3);
          if (gm < M && gn < N && (W == 1 || (r & 1) == 0)) epi.template fetch<ACT, W>(res[k], gm, gn, N, true);
        }
      }
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const auto& rr = res[EPI == EPI_RESIDUAL ? 4 * i + jj : 0];
          const int gm = m0 + wm * Cfg::WM + 16 * i + 4 * g + jj;
          const bool in = gm < M && gn < N;
          float v[1] = {MODE == MODE_TENSOR ? acc[i][j][jj] * s : acc[i][j][jj]};
          epi.pre(v, b);
          if (in) epi.aux(v, gm, gn, N, true);
          if constexpr (ACT == FP8_ACT_SWIGLU) {
            // the up value of an even (gate) column is held by the next lane
            float w[2] = {v[0], __shfl_xor(v[0], 1, 64)};
            if (in && (r & 1) == 0) epi.template out<ACT>(w, gm, gn, N, true, rr);
          } else if (in) {
            epi.template out<ACT>(v, gm, gn, N, true, rr);
          }
        }
    }
  });
  epi.finish(lane, reinterpret_cast<uint32_t*>(smem));
}

}  // namespace sfp8
