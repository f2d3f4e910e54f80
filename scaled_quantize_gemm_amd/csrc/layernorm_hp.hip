// LayerNorm with a high-precision output, and its backward pass.
//
//   mean = sum(x) / cols, var = sum((x - mean)^2) / cols, rs = 1 / sqrt(var + eps)
//   y = (x - mean) rs gamma + beta
//   dx = rs (g - mean(g) - xh mean(g xh)) + dres,  g = dy gamma,  xh = (x - mean) rs
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy
//
// Both are bound by memory: x (and dy, dres) once in, y or dx once out.  A team of W waves holds a row in registers,
// 8-element chunks dealt over its lanes (NCH per lane), so the row is read once; blocks are persistent, each lane
// keeps gamma (and beta) of its columns for the block's lifetime and loads its next row before it works on the
// current one.
//
// Row statistics over W waves in one barrier: each wave reduces its own mean and squared deviations (two passes over
// registers, no cancellation), and the waves' results are merged by  M2 = sum M2_w + n_w (mean_w - mean)^2.
// Backward: a lane's columns are the same for every row of the block, so dgamma and dbeta add up in registers;
// a block's teams join theirs in LDS and write one partial row each, which a second kernel adds up in order.
#include <algorithm>

#include "col_reduce.h"

namespace sfp8 {

constexpr int64_t kLnMaxCols = 32768;

// 8 consecutive elements as loaded.  Rows of odd widths start at any element, so the vectors are loaded and stored at
// the element's alignment (the hardware takes 16 bytes at any address; an unaligned one touches a line more).
template <bool BF16>
struct LnChunk {
  u32x4 w[BF16 ? 1 : 2];
};
template <bool BF16>
struct LnVec;
template <>
struct LnVec<true> {
  typedef u32x4 type __attribute__((aligned(2)));
};
template <>
struct LnVec<false> {
  typedef u32x4 type __attribute__((aligned(4)));
};

// elements c .. c+7 of a row of `cols` (those past its end read as 0)
template <bool BF16, bool TAIL>
__device__ __forceinline__ void ln_load(const void* row, int c, int cols, LnChunk<BF16>& v) {
  if (!TAIL || c + 8 <= cols) {
    typedef typename LnVec<BF16>::type V;
    if constexpr (BF16) {
      v.w[0] = __builtin_nontemporal_load(reinterpret_cast<const V*>(static_cast<const uint16_t*>(row) + c));
    } else {
      const V* p = reinterpret_cast<const V*>(static_cast<const float*>(row) + c);
      v.w[0] = __builtin_nontemporal_load(p);
      v.w[1] = __builtin_nontemporal_load(p + 1);
    }
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = 0u;
      if (c + i < cols) {
        if constexpr (BF16) e[i] = static_cast<const uint16_t*>(row)[c + i];
        else e[i] = static_cast<const uint32_t*>(row)[c + i];
      }
    }
    if constexpr (BF16) {
      v.w[0] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    } else {
      v.w[0] = u32x4{e[0], e[1], e[2], e[3]};
      v.w[1] = u32x4{e[4], e[5], e[6], e[7]};
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void ln_widen(const LnChunk<BF16>& c, float (&v)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    const uint32_t w[8] = {c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w, c.w[1].x, c.w[1].y, c.w[1].z, c.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
}

// 8 values rounded to the output's type
template <bool BF16, bool TAIL>
__device__ __forceinline__ void ln_store(void* row, int c, int cols, const float (&v)[8]) {
  if (!TAIL || c + 8 <= cols) {
    typedef typename LnVec<BF16>::type V;
    if constexpr (BF16) {
      const u32x4 w = {f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                       f32x2_to_bf16x2(v[6], v[7])};
      __builtin_nontemporal_store(w, reinterpret_cast<V*>(static_cast<uint16_t*>(row) + c));
    } else {
      V* p = reinterpret_cast<V*>(static_cast<float*>(row) + c);
      const u32x4 a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      const u32x4 b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
      __builtin_nontemporal_store(a, p);
      __builtin_nontemporal_store(b, p + 1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) {
        if constexpr (BF16) static_cast<uint16_t*>(row)[c + i] = (uint16_t)f32_to_bf16_bits(v[i]);
        else static_cast<float*>(row)[c + i] = v[i];
      }
  }
}

// gamma or beta (fp32 or bf16; null: zeros) of the columns c .. c+7 (aligned; those past the row's end: 0)
template <bool TAIL>
__device__ __forceinline__ void ln_weights(const void* p, int bf16, int c, int cols, float (&v)[8]) {
  if (p == nullptr || c >= cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  } else if (TAIL && c + 8 > cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (c + i < cols)
        v[i] = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[c + i] << 16)
                    : static_cast<const float*>(p)[c + i];
    }
  } else if (bf16) {
    LnChunk<true> w;
    w.w[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + c);
    ln_widen<true>(w, v);
  } else {
    LnChunk<false> w;
    w.w[0] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + c);
    w.w[1] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + c + 4);
    ln_widen<false>(w, v);
  }
}

// sum over the wave, the same in every lane: DPP within rows of 16 lanes, shuffles across them
__device__ __forceinline__ float ln_wave_sum(float v) {
  v += __uint_as_float(dpp_partner<kDppQuadXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_partner<kDppQuadXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_partner<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_partner<kDppMirror>(__float_as_uint(v)));
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// columns of a partial row of dgamma or dbeta: whole 8-column chunks
__host__ __device__ inline int ln_pitch(int64_t cols) { return (int)((cols + 7) & ~7ll); }

// a block's shape for teams of W waves
template <int W>
struct LnBlock {
  static constexpr int kTeams = W >= 8 ? 1 : 8 / W, kThreads = 64 * W * kTeams;
};

template <int W, int NCH, bool XBF, bool YBF, bool TAIL>
__global__ void __launch_bounds__(LnBlock<W>::kThreads) ln_fwd_kernel(const void* x, const void* __restrict__ gamma,
                                                                      const void* __restrict__ beta, int w_bf16,
                                                                      float eps, int64_t rows, int cols, void* y,
                                                                      float* __restrict__ mu,
                                                                      float* __restrict__ rs_out) {
  constexpr int G = LnBlock<W>::kTeams;
  constexpr bool KEEP = NCH <= 2;  // gamma and beta in registers
  constexpr int XB = XBF ? 2 : 4, YB = YBF ? 2 : 4;
  __shared__ float red[2][G][W][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int team = wave / W, w = wave % W;
  int col[NCH];
#pragma unroll
  for (int p = 0; p < NCH; ++p) col[p] = 8 * (lane + 64 * (w + W * p));
  // elements of this wave
  int n_w = 0;
#pragma unroll
  for (int p = 0; p < NCH; ++p) n_w += std::max(0, std::min(512, cols - 512 * (w + W * p)));
  float gam[KEEP ? NCH : 1][8], bet[KEEP ? NCH : 1][8];
  LnChunk<XBF> raw[NCH];
  auto load_row = [&](int64_t row) {
    const char* base = static_cast<const char*>(x) + row * cols * XB;
#pragma unroll
    for (int p = 0; p < NCH; ++p)
      if (col[p] < cols) ln_load<XBF, TAIL>(base, col[p], cols, raw[p]);
  };
  int64_t row = (int64_t)blockIdx.x * G + team;
  const int64_t step = (int64_t)gridDim.x * G;
  if (row < rows) load_row(row);
  if constexpr (KEEP) {
#pragma unroll
    for (int p = 0; p < NCH; ++p) {
      ln_weights<TAIL>(gamma, w_bf16, col[p], cols, gam[p]);
      ln_weights<TAIL>(beta, w_bf16, col[p], cols, bet[p]);
    }
  }
  int buf = 0;
  // the block's teams run in step (row - team is the block's)
  for (; row - team < rows; row += step, buf ^= 1) {
    const bool live = row < rows;
    float v[NCH][8], sum = 0.0f;
#pragma unroll
    for (int p = 0; p < NCH; ++p) {
      if (col[p] < cols) {
        ln_widen<XBF>(raw[p], v[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[p][i];
      }
    }
    if (row + step < rows) load_row(row + step);
    float mean = ln_wave_sum(sum) / (float)std::max(n_w, 1), m2 = 0.0f;
#pragma unroll
    for (int p = 0; p < NCH; ++p)
      if (col[p] < cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!TAIL || col[p] + i < cols) {
            const float d = v[p][i] - mean;
            m2 += d * d;
          }
      }
    m2 = ln_wave_sum(m2);
    if constexpr (W > 1) {
      if (lane == 0) {
        red[buf][team][w][0] = mean;
        red[buf][team][w][1] = m2;
      }
      __syncthreads();
      float total = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        int n_k = 0;
#pragma unroll
        for (int p = 0; p < NCH; ++p) n_k += std::max(0, std::min(512, cols - 512 * (k + W * p)));
        total += red[buf][team][k][0] * (float)n_k;
      }
      mean = total / (float)cols;
      m2 = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        int n_k = 0;
#pragma unroll
        for (int p = 0; p < NCH; ++p) n_k += std::max(0, std::min(512, cols - 512 * (k + W * p)));
        const float d = red[buf][team][k][0] - mean;
        m2 += red[buf][team][k][1] + (n_k > 0 ? d * d * (float)n_k : 0.0f);
      }
    }
    const float rs = 1.0f / sqrtf(m2 / (float)cols + eps);
    if (!live) continue;
    if (lane == 0 && w == 0) {
      if (mu != nullptr) mu[row] = mean;
      if (rs_out != nullptr) rs_out[row] = rs;
    }
    char* out = static_cast<char*>(y) + row * cols * YB;
#pragma unroll
    for (int p = 0; p < NCH; ++p) {
      if (col[p] >= cols) continue;
      float g[8], b[8], o[8];
      if constexpr (!KEEP) {
        ln_weights<TAIL>(gamma, w_bf16, col[p], cols, g);
        ln_weights<TAIL>(beta, w_bf16, col[p], cols, b);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = (v[p][i] - mean) * rs;
        const float gi = KEEP ? gam[KEEP ? p : 0][i] : g[i], bi = KEEP ? bet[KEEP ? p : 0][i] : b[i];
        o[i] = fmaf(t, gi, bi);
      }
      ln_store<YBF, TAIL>(out, col[p], cols, o);
    }
  }
}

template <int W, int NCH, bool XBF, bool DBF, bool TAIL>
__global__ void __launch_bounds__(LnBlock<W>::kThreads) ln_bwd_kernel(const void* dy, const void* __restrict__ x,
                                                                      const void* __restrict__ gamma, int w_bf16,
                                                                      const float* __restrict__ mu,
                                                                      const float* __restrict__ rsig, const void* dres,
                                                                      int64_t rows, int cols, void* dx,
                                                                      float* __restrict__ part,
                                                                      float* __restrict__ dgamma,
                                                                      float* __restrict__ dbeta) {
  constexpr int G = LnBlock<W>::kTeams;
  constexpr bool KEEP = NCH <= 2;
  constexpr int XB = XBF ? 2 : 4, DB = DBF ? 2 : 4;
  // row sums; at the end the teams' column sums (one team: none)
  __shared__ float red[2][G][W][2];
  __shared__ __attribute__((aligned(16))) float join[G > 1 ? 2 * 512 * W * NCH : 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int team = wave / W, w = wave % W;
  int col[NCH];
#pragma unroll
  for (int p = 0; p < NCH; ++p) col[p] = 8 * (lane + 64 * (w + W * p));
  float gam[KEEP ? NCH : 1][8], dg[NCH][8], db[NCH][8];
#pragma unroll
  for (int p = 0; p < NCH; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[p][i] = db[p][i] = 0.0f;
  LnChunk<XBF> rx[NCH], rr[NCH];
  LnChunk<DBF> rd[NCH];
  float m_next = 0.0f, s_next = 0.0f;
  auto load_row = [&](int64_t row) {
    const char* bx = static_cast<const char*>(x) + row * cols * XB;
    const char* bd = static_cast<const char*>(dy) + row * cols * DB;
    m_next = mu[row];
    s_next = rsig[row];
#pragma unroll
    for (int p = 0; p < NCH; ++p)
      if (col[p] < cols) {
        ln_load<XBF, TAIL>(bx, col[p], cols, rx[p]);
        ln_load<DBF, TAIL>(bd, col[p], cols, rd[p]);
        if (dres != nullptr)
          ln_load<XBF, TAIL>(static_cast<const char*>(dres) + row * cols * XB, col[p], cols, rr[p]);
      }
  };
  int64_t row = (int64_t)blockIdx.x * G + team;
  const int64_t step = (int64_t)gridDim.x * G;
  if (row < rows) load_row(row);
  if constexpr (KEEP) {
#pragma unroll
    for (int p = 0; p < NCH; ++p) ln_weights<TAIL>(gamma, w_bf16, col[p], cols, gam[p]);
  }
  int buf = 0;
  for (; row - team < rows; row += step, buf ^= 1) {
    const bool live = row < rows;
    const float m = m_next, rs = s_next;
    float xh[NCH][8], g[NCH][8], res[NCH][8], s1 = 0.0f, s2 = 0.0f;
    if (live) {
#pragma unroll
      for (int p = 0; p < NCH; ++p)
        if (col[p] < cols) {
          float d[8], gw[8];
          ln_widen<XBF>(rx[p], xh[p]);
          ln_widen<DBF>(rd[p], d);
          if (dres != nullptr) ln_widen<XBF>(rr[p], res[p]);
          if constexpr (!KEEP) ln_weights<TAIL>(gamma, w_bf16, col[p], cols, gw);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // past the row's end dy reads as 0 and drops out of every sum
            xh[p][i] = (xh[p][i] - m) * rs;
            g[p][i] = d[i] * (KEEP ? gam[KEEP ? p : 0][i] : gw[i]);
            dg[p][i] = fmaf(d[i], xh[p][i], dg[p][i]);
            db[p][i] += d[i];
            s1 += g[p][i];
            s2 = fmaf(g[p][i], xh[p][i], s2);
          }
        }
    }
    if (row + step < rows) load_row(row + step);
    s1 = ln_wave_sum(s1);
    s2 = ln_wave_sum(s2);
    if constexpr (W > 1) {
      if (lane == 0) {
        red[buf][team][w][0] = s1;
        red[buf][team][w][1] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        s1 += red[buf][team][k][0];
        s2 += red[buf][team][k][1];
      }
    }
    s1 /= (float)cols;
    s2 /= (float)cols;
    if (!live) continue;
    char* out = static_cast<char*>(dx) + row * cols * XB;
#pragma unroll
    for (int p = 0; p < NCH; ++p) {
      if (col[p] >= cols) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = rs * (g[p][i] - s1 - xh[p][i] * s2);
        if (dres != nullptr) o[i] += res[p][i];
      }
      ln_store<XBF, TAIL>(out, col[p], cols, o);
    }
  }
  // the teams' column sums, added one team after the other, the last one to the block's partial row [2][pitch], or
  // (part null: the only block) to dgamma and dbeta
  const int pitch = ln_pitch(cols);
  float* mine = part + (int64_t)blockIdx.x * 2 * pitch;
#pragma unroll 1
  for (int t = 0; t < G; ++t) {
    if (team == t) {
#pragma unroll
      for (int p = 0; p < NCH; ++p) {
        if (col[p] >= cols) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            float(&v)[8] = h == 0 ? dg[p] : db[p];
            float4 sum = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            if constexpr (G > 1) {
              float4* at = reinterpret_cast<float4*>(join + h * 512 * W * NCH + col[p] + i);
              if (t > 0) {
                const float4 o = *at;
                sum = make_float4(sum.x + o.x, sum.y + o.y, sum.z + o.z, sum.w + o.w);
              }
              if (t < G - 1) *at = sum;
            }
            if (t < G - 1) continue;
            if (part != nullptr) {
              *reinterpret_cast<float4*>(mine + h * pitch + col[p] + i) = sum;
            } else if (float* out = h == 0 ? dgamma : dbeta) {
              const float o[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!TAIL || col[p] + i + k < cols) out[col[p] + i + k] = o[k];
            }
          }
      }
    }
    if constexpr (G > 1) __syncthreads();
  }
}

// f(W, NCH) with the team that holds a row of `cols`.  Forward: up to 4 chunks per lane, few waves per barrier (8192 x 4096
// bf16: 27 us with 2 x 4, 30 with 4 x 2, 28-32 with 8 x 1).  Backward, whose lanes hold three rows and two sums per chunk:
// as few chunks as 8 waves allow (8192 x 4096 with dres: 47 us with 8 x 1 or 4 x 2, 69 with 2 x 4).
template <bool BWD, class F>
static void ln_shape(int64_t cols, F&& f) {
  using std::integral_constant;
  auto g = [&](auto w, auto n) { f(w, n); };
#define SFP8_LN_SHAPE(W, N) g(integral_constant<int, W>{}, integral_constant<int, N>{})
  if (cols <= 512) SFP8_LN_SHAPE(1, 1);
  else if (cols <= 1024) SFP8_LN_SHAPE(BWD ? 2 : 1, BWD ? 1 : 2);
  else if (cols <= 2048) SFP8_LN_SHAPE(BWD ? 4 : 1, BWD ? 1 : 4);
  else if (cols <= 4096) SFP8_LN_SHAPE(BWD ? 8 : 2, BWD ? 1 : 4);
  else if (cols <= 8192) SFP8_LN_SHAPE(BWD ? 8 : 4, BWD ? 2 : 4);
  else if (cols <= 16384) SFP8_LN_SHAPE(BWD ? 16 : 8, BWD ? 2 : 4);
  else SFP8_LN_SHAPE(16, 4);
#undef SFP8_LN_SHAPE
}

// f(bool a, bool b, bool c) with three run-time truth values as constants
template <class F>
static void ln_types(bool a, bool b, bool c, F&& f) {
  using T = std::true_type;
  using N = std::false_type;
  auto g = [&](auto x, auto y) {
    if (c) f(x, y, T{});
    else f(x, y, N{});
  };
  if (a) {
    if (b) g(T{}, T{});
    else g(T{}, N{});
  } else {
    if (b) g(N{}, T{});
    else g(N{}, N{});
  }
}

// blocks of the backward: at most 256, one per CU, each with a partial row of dgamma and dbeta (512 took 6 us more on
// 8192 x 4096: twice the partial rows to write and join); up to 4 rows per team one block does it all, without the
// partial row, the workspace and the second launch (16 x 768: a call 13.9 us, 6.7 in a graph; 17 x 768, with them: 18.2 and
// 6.2)
constexpr int64_t kLnBwdBlocks = 256, kLnAloneRows = 4;
static int64_t ln_bwd_blocks(int64_t rows, int64_t cols) {
  int64_t teams = 1;
  ln_shape<true>(cols, [&](auto w, auto) { teams = LnBlock<decltype(w)::value>::kTeams; });
  if (rows <= kLnAloneRows * teams) return rows > 0;
  return std::min(kLnBwdBlocks, (rows + teams - 1) / teams);
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
  const int wb = w_dtype == HP_BF16, c = (int)cols;
  ln_shape<false>(cols, [&](auto wc, auto nc) {
    constexpr int W = decltype(wc)::value, NCH = decltype(nc)::value;
    using B = LnBlock<W>;
    ln_types(x_dtype == HP_BF16, y_dtype == OUT_BF16, cols % 8 != 0, [&](auto xb, auto yb, auto tail) {
      // at most 4 blocks per CU, and beyond one per CU at least two rows per team (8192 x 1024: 512 blocks 8.1 us,
      // 1024 blocks 9.8)
      const int64_t groups = (rows + B::kTeams - 1) / B::kTeams, cus = device_cus();
      const int64_t blocks = std::min(groups, std::max(cus, std::min(4 * cus, groups / 2)));
      hipLaunchKernelGGL((ln_fwd_kernel<W, NCH, decltype(xb)::value, decltype(yb)::value, decltype(tail)::value>),
                         dim3((unsigned)blocks), dim3(B::kThreads), 0, st, x, gamma, beta, wb, eps, rows, c, y, mu,
                         rsigma);
    });
  });
  return check_launch(what);
}

extern "C" size_t fp8_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows >= (1ll << 31) || cols < 0 || cols > kLnMaxCols) return 0;
  const int64_t blocks = ln_bwd_blocks(rows, cols);
  return blocks <= 1 ? 0 : (size_t)blocks * 2 * (size_t)ln_pitch(cols) * sizeof(float);
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
  const int64_t blocks = ln_bwd_blocks(rows, cols);
  float* part = blocks == 1 ? nullptr : static_cast<float*>(workspace);
  if (rows > 0) {
    SFP8_REQUIRE(dy != nullptr && x != nullptr && gamma != nullptr && mu != nullptr && rsigma != nullptr && dx != nullptr,
                 FP8_ERR_ARG, "%s: null dy, x, gamma, mu, rsigma or dx", what);
    SFP8_REQUIRE(aligned16(dy) && aligned16(x) && aligned16(gamma) && aligned16(dres) && aligned16(dx), FP8_ERR_ARG,
                 "%s: dy, x, gamma, dres, dx must be 16-byte aligned", what);
    SFP8_REQUIRE(aligned4(mu) && aligned4(rsigma), FP8_ERR_ARG, "%s: misaligned mu / rsigma", what);
    SFP8_REQUIRE(dx != dy || dy_dtype == x_dtype, FP8_ERR_ARG, "%s: dx may be dy only where dy has x's type", what);
    SFP8_REQUIRE(dx != x, FP8_ERR_ARG, "%s: dx may not be x", what);
    const size_t need = fp8_layernorm_backward_workspace(rows, cols);
    SFP8_REQUIRE(need == 0 || (workspace != nullptr && aligned16(workspace) && workspace_bytes >= need), FP8_ERR_ARG,
                 "%s: workspace of %zu bytes, 16-byte aligned, needed (%zu given)", what, need, workspace_bytes);
    ln_shape<true>(cols, [&](auto wc, auto nc) {
      constexpr int W = decltype(wc)::value, NCH = decltype(nc)::value;
      ln_types(x_dtype == HP_BF16, dy_dtype == HP_BF16, cols % 8 != 0, [&](auto xb, auto db, auto tail) {
        hipLaunchKernelGGL((ln_bwd_kernel<W, NCH, decltype(xb)::value, decltype(db)::value, decltype(tail)::value>),
                           dim3((unsigned)blocks), dim3(LnBlock<W>::kThreads), 0, st, dy, x, gamma, wb, mu, rsigma,
                           dres, rows, c, dx, part, dgamma, dbeta);
      });
    });
    const int rc = check_launch(what);
    if (rc != FP8_OK) return rc;
  }
  if (blocks == 1) return FP8_OK;
  launch_col_reduce(part, (int)blocks, 2, ln_pitch(cols), cols, dgamma, dbeta, st);
  return check_launch(what);
}
