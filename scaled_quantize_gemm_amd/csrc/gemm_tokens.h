// The FP8 GEMM for a few rows (a decoding step's tokens) with the residual epilogue: bound by reading the weights
// B [N][K] once, at most 64 rows of A against them.
//
// A block owns NT tiles of 16 columns of C and all rows (MT tiles of 16); its NW waves split K, wave w taking the 128-deep
// steps w, w + NW, ...: 16 x 16 x 128 MFMAs on fragments loaded straight from memory (each lane's two 16-byte pieces
// of a row; a wave's pieces of a step are whole 128-byte lines), U steps of loads in flight per wave.  No LDS on the way
// in: nothing is used twice but A, which the caches hold.  The waves' sums meet in LDS and are added in the order of
// the waves; one thread per output runs the epilogue.
#pragma once

#include "gemm_common.h"

namespace sfp8 {

template <int MODE, int FA, int OUT, int MT, int NT, int NW, int U>
__global__ void __launch_bounds__(64 * NW) gemm_tokens_kernel(const uint8_t* __restrict__ A,
                                                                     const uint8_t* __restrict__ B,
                                                                     const void* __restrict__ sa_p,
                                                                     const void* __restrict__ sb_p, const EpiParams ep,
                                                                     int M, int N, int K) {
  constexpr int FB = FP8_E4M3, COLS = 16 * NT;
  __shared__ float red[NW][MT * 16 * COLS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int n0 = blockIdx.x * COLS, nk = K / 128;
  // rows and columns past the end repeat the last one; their results are dropped
  int gn[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) gn[c] = n0 + 16 * c + r < N ? n0 + 16 * c + r : N - 1;
  int gm[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) gm[i] = 16 * i + r < M ? 16 * i + r : M - 1;
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[i][c] = v4f{0.f, 0.f, 0.f, 0.f};

  auto frag = [&](const uint8_t* row, int ks) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(row + (size_t)ks * 128 + 16 * g);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(row + (size_t)ks * 128 + 64 + 16 * g);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  for (int k0 = wave; k0 < nk; k0 += U * NW) {
    v8i fb[U][NT], fa[U][MT];
    // scales of a step: MX codes of A and B; blockwise the rows' scales and the columns' (or the block's)
    int ea[U][MT], eb[U][NT];
    float sa[U][MT][4], sb[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ks = k0 + u * NW;
      if (ks >= nk) continue;
#pragma unroll
      for (int c = 0; c < NT; ++c) fb[u][c] = frag(B + (size_t)gn[c] * K, ks);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[u][i] = frag(A + (size_t)gm[i] * K, ks);
      if constexpr (MODE == MODE_MX) {
#pragma unroll
        for (int c = 0; c < NT; ++c) eb[u][c] = static_cast<const uint8_t*>(sb_p)[(size_t)(4 * ks + g) * N + gn[c]];
#pragma unroll
        for (int i = 0; i < MT; ++i) ea[u][i] = static_cast<const uint8_t*>(sa_p)[(size_t)(4 * ks + g) * M + gm[i]];
      } else if constexpr (MODE != MODE_TENSOR) {
        const float* s = static_cast<const float*>(sb_p);
        // a block's columns lie within one weight block
#pragma unroll
        for (int c = 0; c < NT; ++c)
          sb[u][c] = MODE == MODE_BLOCK ? s[(size_t)(n0 / 128) * nk + ks] : s[(size_t)ks * N + gn[c]];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int m = 16 * i + 4 * g + j;
            sa[u][i][j] = static_cast<const float*>(sa_p)[(size_t)ks * M + (m < M ? m : M - 1)];
          }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * NW >= nk) continue;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          v4f& d = acc[i][c];
          if constexpr (MODE == MODE_TENSOR) {
            d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[u][i], fb[u][c], d, FA, FB, 0, 0, 0, 0);
          } else if constexpr (MODE == MODE_MX) {
            d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[u][i], fb[u][c], d, FA, FB, 0, ea[u][i], 0, eb[u][c]);
          } else {
            const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa[u][i], fb[u][c], v4f{0.f, 0.f, 0.f, 0.f}, FA,
                                                                           FB, 0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = fmaf(p[j], sa[u][i][j] * sb[u][c], d[j]);
          }
        }
    }
  }
  // lane (g, r) holds rows 16 i + 4 g + j of column r
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[wave][(16 * i + 4 * g + j) * COLS + 16 * c + r] = acc[i][c][j];
  __syncthreads();
  float s = 1.0f;
  if constexpr (MODE == MODE_TENSOR) s = *static_cast<const float*>(sa_p) * *static_cast<const float*>(sb_p);
  Epilogue<OUT, EPI_RESIDUAL> epi(ep);
  epi.with_act([&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
    // whole waves: SwiGLU's column pairs are neighbouring lanes
    for (int t = threadIdx.x; t < MT * 16 * COLS; t += 64 * NW) {
      float v[1] = {0.0f}, b[1];
#pragma unroll
      for (int w = 0; w < NW; ++w) v[0] += red[w][t];
      if constexpr (MODE == MODE_TENSOR) v[0] *= s;
      const int m = t / COLS, n = n0 + t % COLS;
      const bool in = m < M && n < N;
      constexpr int W = ACT == FP8_ACT_SWIGLU ? 2 : 1;
      typename Epilogue<OUT, EPI_RESIDUAL>::template Run<ACT, W> res;
      const bool stores = in && (W == 1 || (n & 1) == 0);
      if (stores) epi.template fetch<ACT, W>(res, m, n, N, true);
      epi.template bias<1>(n, N, b);
      epi.pre(v, b);
      if constexpr (ACT == FP8_ACT_SWIGLU) {
        float w[2] = {v[0], __shfl_xor(v[0], 1, 64)};
        if (stores) epi.template out<ACT>(w, m, n, N, true, res);
      } else if (stores) {
        epi.template out<ACT>(v, m, n, N, true, res);
      }
    }
  });
}

// the problems it takes: up to 64 rows, up to 32 per tensor over wide weights, whose tiles of the large kernels fill the
// chip (4 .. 64 rows, us here / there: per tensor 4096 x 7168 8.1-18.5 / 21-23.5, 14336 x 4096 at 32 rows 15.6 / 18.1
// and at 64 21.3 / 18.6; blockwise 4096 x 7168 9.4-20.7 / 40-48; MX 8.8-19.2 / 63-78)
constexpr int kTokRows = 64, kTokRowsWide = 32, kTokWideN = 12288;

template <int MODE>
static bool tokens_apply(int M, int N) {
  // (a launch holds less than 2^32 threads)
  return M <= (MODE == MODE_TENSOR && N >= kTokWideN ? kTokRowsWide : kTokRows) && N <= (1 << 24);
}

// Tiles of 16 columns per block: as many as leave about a block per CU, so that A is read by fewer blocks (14336 x 4096
// at 16 rows: 17.9 us with 1, 14.4 with 2, 12.8 with 4; 4096 x 7168: 8.9, 11.9, 18.0).  Waves per block and steps in
// flight per wave matter little (within 5%) and follow from the registers.
template <int MODE, int FA, int OUT, int MT>
static int launch_tokens_rows(const uint8_t* A, const uint8_t* B, const void* sa, const void* sb, const EpiParams& ep,
                              int M, int N, int K, hipStream_t st, const char* what) {
  constexpr int U = MT == 4 ? 1 : 2;
#define SFP8_TOK(NT, NW)                                                                                             \
  hipLaunchKernelGGL((gemm_tokens_kernel<MODE, FA, OUT, MT, NT, NW, U>),                                             \
                     dim3((unsigned)((N + 16 * NT - 1) / (16 * NT))), dim3(64 * NW), 0, st, A, B, sa, sb, ep, M, N, K)
  if (N >= kTokWideN) SFP8_TOK(4, 8);
  else if (N >= kTokWideN / 2) SFP8_TOK(2, 8);
  else SFP8_TOK(1, 16);
#undef SFP8_TOK
  return check_launch(what);
}

template <int MODE, int FA, int OUT>
static int launch_tokens(const uint8_t* A, const uint8_t* B, const void* sa, const void* sb, const EpiParams& ep, int M,
                         int N, int K, hipStream_t st, const char* what) {
  if (M <= 16) return launch_tokens_rows<MODE, FA, OUT, 1>(A, B, sa, sb, ep, M, N, K, st, what);
  if (M <= 32) return launch_tokens_rows<MODE, FA, OUT, 2>(A, B, sa, sb, ep, M, N, K, st, what);
  return launch_tokens_rows<MODE, FA, OUT, 4>(A, B, sa, sb, ep, M, N, K, st, what);
}

}  // namespace sfp8
