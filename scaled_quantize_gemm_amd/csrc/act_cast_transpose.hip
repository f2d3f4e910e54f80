// Activation (forward) and activation gradient (backward), cast to FP8 with the transpose and, backward,
// the bias gradient.
//
// forward   h = gelu(v) or silu(v[2f]) v[2f+1]
// backward  d = dh act'(v): GELU dh (Phi(v) + v phi(v)); SwiGLU (interleaved columns, s = sigmoid(g))
//           d[2f] = dh u s (1 + g (1 - s)), d[2f+1] = dh g s;  dbias = sum_rows d
// and the result goes to FP8 under the cast rules of quantize.hip, per tensor (delayed scale, amax into a
// slot) or in 1x128 runs (its own for q and for the transposed copy).
//
// Bound by memory: pre and dh once in, two copies of the codes out.  One 512-thread block per 128 x 128 tile of the
// result: thread t computes rows t/16 + 32p (p = 0..3), columns 8(t%16)..+8, from 16-byte loads, casts them, writes q,
// and puts the codes for qT into an LDS tile (dword pitch 33) that leaves with 4x4 byte transposes, 128 contiguous bytes of a
// qT row per 32 lanes.  Per tensor the scale is known beforehand, so a value is cast as soon as it is computed
// and a block's next tile is loaded before it transposes the current one; in 1x128 runs the thread's 32 values wait in
// registers for the row and column maxima.  The bias gradient's column sums go through lane exchanges and LDS
// to one partial row per tile row, joined by a second kernel in order.
//
// Any size and alignment: vectors are loaded and stored at the element's alignment (the hardware takes them at any
// address), tiles at the edge test their rows and chunks, and a row's last partial chunk goes by element.
#include <algorithm>

#include "act_math.h"
#include "col_reduce.h"
#include "quant_rules.h"

namespace sfp8 {

constexpr int kActTile = 128, kActPitch = 33;
// what a kernel computes from its inputs
enum { ACT_FWD_GELU = 0, ACT_FWD_SWIGLU = 1, ACT_BWD_NONE = 2, ACT_BWD_GELU = 3, ACT_BWD_SWIGLU = 4 };

// N consecutive elements as loaded (N = 4, 8, 16), kept packed until the arithmetic
template <bool BF16, int N>
struct ActRaw {
  static constexpr int kWords = BF16 ? N / 2 : N;
  uint32_t w[kWords];
};

template <int N>
struct ActVec;
template <>
struct ActVec<2> {
  typedef u32x2 type __attribute__((aligned(2)));
};
template <>
struct ActVec<4> {
  typedef u32x4 type __attribute__((aligned(2)));
};

// elements c .. c+N-1 of a row of `cols` at p (those past its end read as 0)
template <bool BF16, int N, bool EDGE>
__device__ __forceinline__ void act_load(const void* row, int64_t c, int64_t cols, ActRaw<BF16, N>& r) {
  constexpr int W = ActRaw<BF16, N>::kWords, V = W < 4 ? W : 4;
  if (!EDGE || c + N <= cols) {
    const char* p = static_cast<const char*>(row) + c * (BF16 ? 2 : 4);
    typedef typename ActVec<V>::type T;
#pragma unroll
    for (int i = 0; i < W / V; ++i) {
      const auto v = __builtin_nontemporal_load(reinterpret_cast<const T*>(p) + i);
#pragma unroll
      for (int j = 0; j < V; ++j) r.w[V * i + j] = v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < cols) {
        if constexpr (BF16) r.w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(row)[c + i] << (16 * (i & 1));
        else r.w[i] = static_cast<const uint32_t*>(row)[c + i];
      }
  }
}

template <bool BF16, int N>
__device__ __forceinline__ float act_elem(const ActRaw<BF16, N>& r, int i) {
  if constexpr (BF16) return (i & 1) ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
  else return __uint_as_float(r.w[i]);
}

// the inputs of 8 adjacent results of a row
template <int OP, bool BF16>
struct ActIn {
  static constexpr bool kPre = OP != ACT_BWD_NONE, kDh = OP >= ACT_BWD_NONE;
  static constexpr int kPreN = OP == ACT_FWD_SWIGLU ? 16 : 8, kDhN = OP == ACT_BWD_SWIGLU ? 4 : 8;
  ActRaw<BF16, kPreN> pre;
  ActRaw<BF16, kDhN> dh;

  // results (row, c .. c+7) of [rows][cols]
  template <bool EDGE>
  __device__ __forceinline__ void load(const void* dhp, const void* prep, int64_t row, int64_t c, int64_t cols) {
    constexpr int E = BF16 ? 2 : 4;
    if constexpr (kPre) {
      constexpr int64_t f = kPreN / 8;
      act_load<BF16, kPreN, EDGE>(static_cast<const char*>(prep) + row * cols * f * E, c * f, cols * f, pre);
    }
    if constexpr (kDh) {
      constexpr int64_t f = 8 / kDhN;
      act_load<BF16, kDhN, EDGE>(static_cast<const char*>(dhp) + row * (cols / f) * E, c / f, cols / f, dh);
    }
  }
  // zero inputs: every result 0
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < ActRaw<BF16, kPreN>::kWords; ++i) pre.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < ActRaw<BF16, kDhN>::kWords; ++i) dh.w[i] = 0u;
  }
  __device__ __forceinline__ void results(float (&v)[8]) const {
    if constexpr (OP == ACT_FWD_GELU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_gelu(act_elem(pre, i));
    } else if constexpr (OP == ACT_FWD_SWIGLU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_swiglu(act_elem(pre, 2 * i), act_elem(pre, 2 * i + 1));
    } else if constexpr (OP == ACT_BWD_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_elem(dh, i);
    } else if constexpr (OP == ACT_BWD_GELU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_elem(dh, i) * act_gelu_grad(act_elem(pre, i));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        act_swiglu_grad(act_elem(dh, i), act_elem(pre, 2 * i), act_elem(pre, 2 * i + 1), v[2 * i], v[2 * i + 1]);
    }
  }
};

// max of |a|, |b|, |c| that keeps a NaN (one v_maximum3_f32); as bits NaN is above everything
__device__ __forceinline__ float act_max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b)),
                                       __builtin_fabsf(c));
}
__device__ __forceinline__ uint32_t act_amax8(const float (&v)[8]) {
  const float m = act_max3(act_max3(v[0], v[1], v[2]), v[3], v[4]);
  return abs_bits(act_max3(act_max3(m, v[5], v[6]), v[7], v[7]));
}

// Sum (or max) over the wave's four 16-lane rows of each of 8 values, spread out: lane 16 k + c gets those of its column
// group c for the elements 2k and 2k + 1.  Each swap exchanges half of one register with half of another, so that
// one addition serves two elements: 6 swaps and 6 additions for 8 values.
template <class F>
__device__ __forceinline__ void act_rows4(const float (&v)[8], float (&o)[2], F&& f) {
  float r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 4]), false, false);
    r[k] = f(__uint_as_float(x[0]), __uint_as_float(x[1]));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(r[k]), __float_as_uint(r[k + 2]), false, false);
    o[k] = f(__uint_as_float(x[0]), __uint_as_float(x[1]));
  }
}

// 8 values under 8 scales.  CLAMP: saturating; without, for scales that map the largest of the values to fmax (one
// rounding of the product past it still converts to fmax)
template <int FMT, bool CLAMP>
__device__ __forceinline__ u32x2 act_cast8(const float (&v)[8], const float (&s)[8], uint32_t amax_bits) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v[i] * s[i];
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* y = x + 4 * h;
    if (CLAMP || amax_bits >= 0x7F800000u) {
      w[h] = cvt4<FMT>(y[0], y[1], y[2], y[3]);
    } else if constexpr (FMT == FP8_E4M3) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    } else {
      const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], 0, false);
      w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], lo, true);
    }
  }
  if (amax_bits > 0x7F800000u) {
    w[0] = patch_nan4(w[0], &v[0]);
    w[1] = patch_nan4(w[1], &v[4]);
  }
  return u32x2{w[0], w[1]};
}

template <int OP, int FMT, bool BF16, bool TILE, bool EDGE>
__global__ void __launch_bounds__(512) act_ct_kernel(const void* __restrict__ dh, const void* __restrict__ pre,
                                                     int64_t rows, int64_t cols, const float* __restrict__ scale_p,
                                                     uint32_t* __restrict__ amax_slot, uint8_t* __restrict__ q,
                                                     float* __restrict__ q_sinv, uint8_t* __restrict__ qT,
                                                     float* __restrict__ qT_sinv, float* __restrict__ part) {
  typedef u32x2 q_t __attribute__((aligned(1)));
  typedef uint32_t qt_t __attribute__((aligned(1)));
  static_assert(!(TILE && EDGE), "1x128 runs need whole tiles");
  __shared__ uint32_t lds[kActTile * kActPitch];
  __shared__ float csum[8][kActTile];
  __shared__ float cred[8][kActTile];
  __shared__ float cscale[kActTile];
  __shared__ uint32_t not_finite;
  const int64_t nkb = (cols + kActTile - 1) / kActTile, nrb = (rows + kActTile - 1) / kActTile, ntiles = nkb * nrb;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int r16 = t >> 4, cg = t & 15;
  // tiles in bands of 8 tile rows, walked column by column: the blocks in flight write 1 KB runs of a qT row
  auto tile_rc = [&](int64_t ix, int64_t& rb, int64_t& kb) {
    constexpr int64_t SR = 8;
    const int64_t band = ix / (SR * nkb), first = band * SR;
    const int64_t h = nrb - first < SR ? nrb - first : SR;
    const int64_t in = ix - band * SR * nkb;
    rb = first + in % h;
    kb = in / h;
  };
  ActIn<OP, BF16> in[4];
  auto load_tile = [&](int64_t ix) {
    int64_t rb, kb;
    tile_rc(ix, rb, kb);
    const int64_t c = kb * kActTile + cg * 8;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t r = rb * kActTile + r16 + 32 * p;
      if (!EDGE || (r < rows && c < cols)) in[p].template load<EDGE>(dh, pre, r, c, cols);
      else in[p].zero();
    }
  };
  float s8[8];
  if constexpr (!TILE) {
    const float s = *scale_p;
#pragma unroll
    for (int e = 0; e < 8; ++e) s8[e] = s;
  }
  uint32_t amax_acc = 0;
  if constexpr (!TILE) load_tile(blockIdx.x);
  for (int64_t ix = blockIdx.x; ix < ntiles; ix += gridDim.x) {
    if (ix != (int64_t)blockIdx.x) __syncthreads();  // the previous tile's transpose is done with the LDS
    if constexpr (TILE) load_tile(ix);
    int64_t rb, kb;
    tile_rc(ix, rb, kb);
    const int64_t r0 = rb * kActTile, c0 = kb * kActTile;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    // q codes of row r16 + 32p at the tile's columns 8 cg
    auto store_q = [&](int p, u32x2 w) {
      const int64_t r = r0 + r16 + 32 * p, c = c0 + cg * 8;
      uint8_t* at = q + r * cols + c;
      if (!EDGE || (r < rows && c + 8 <= cols)) {
        __builtin_nontemporal_store(w, reinterpret_cast<q_t*>(at));
      } else if (r < rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < cols) at[i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
      }
    };
    if constexpr (!TILE) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float v[8];
        in[p].results(v);
        const uint32_t m = act_amax8(v);
        amax_acc = amax_acc > m ? amax_acc : m;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];
        const u32x2 w = act_cast8<FMT, true>(v, s8, m);
        store_q(p, w);
        lds[(r16 + 32 * p) * kActPitch + cg * 2] = w.x;
        lds[(r16 + 32 * p) * kActPitch + cg * 2 + 1] = w.y;
      }
      if (ix + gridDim.x < ntiles) load_tile(ix + gridDim.x);
    } else {
      float v[4][8], srow[4], cm[8], co[2];
      if (t == 0) not_finite = 0u;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        in[p].results(v[p]);
        float si;
        current_scale<FMT>(group_max_u32<16>(act_amax8(v[p])), srow[p], si);
        if (cg == 0) q_sinv[kb * rows + r0 + r16 + 32 * p] = si;  // [cols/128][rows]
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[p][e];
      }
      // column runs: this thread's 4 rows, the wave's 4 lane groups, then the 8 waves
#pragma unroll
      for (int e = 0; e < 8; ++e) cm[e] = act_max3(act_max3(v[0][e], v[1][e], v[2][e]), v[3][e], v[3][e]);
      act_rows4(cm, co, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
      *reinterpret_cast<float2*>(&cred[wave][cg * 8 + 2 * (lane >> 4)]) = make_float2(co[0], co[1]);
      __syncthreads();
      if (t < kActTile) {
        uint32_t c = __float_as_uint(cred[0][t]);
#pragma unroll
        for (int w = 1; w < 8; ++w) c = c > __float_as_uint(cred[w][t]) ? c : __float_as_uint(cred[w][t]);
        float sc, si;
        current_scale<FMT>(c, sc, si);
        cscale[t] = sc;
        if (c >= 0x7F800000u) not_finite = 0x7F800001u;
        qT_sinv[rb * cols + c0 + t] = si;  // [rows/128][cols]
      }
      __syncthreads();
      // an infinity or NaN somewhere in the tile: its runs have scale 1, and the casts clamp and rewrite NaN
      const uint32_t bad = not_finite;
      float scol[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) scol[e] = cscale[cg * 8 + e];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float sr[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sr[e] = srow[p];
        store_q(p, act_cast8<FMT, false>(v[p], sr, bad));
        const u32x2 w = act_cast8<FMT, false>(v[p], scol, bad);
        lds[(r16 + 32 * p) * kActPitch + cg * 2] = w.x;
        lds[(r16 + 32 * p) * kActPitch + cg * 2 + 1] = w.y;
      }
    }
    if (part != nullptr) {
      float so[2];
      act_rows4(sum, so, [](float a, float b) { return a + b; });
      *reinterpret_cast<float2*>(&csum[wave][cg * 8 + 2 * (lane >> 4)]) = make_float2(so[0], so[1]);
    }
    __syncthreads();
    if (part != nullptr && t < kActTile && (!EDGE || c0 + t < cols)) {
      float a = csum[0][t];
#pragma unroll
      for (int w = 1; w < 8; ++w) a += csum[w][t];
      part[rb * cols + c0 + t] = a;
    }
    // transpose: 4 source rows x 4 source columns per dword quad
    const int rg = t & 31, cgt = t >> 5;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cq = cgt + 16 * h;  // columns 4cq .. 4cq+3 of the tile
      const uint32_t d0 = lds[(4 * rg + 0) * kActPitch + cq];
      const uint32_t d1 = lds[(4 * rg + 1) * kActPitch + cq];
      const uint32_t d2 = lds[(4 * rg + 2) * kActPitch + cq];
      const uint32_t d3 = lds[(4 * rg + 3) * kActPitch + cq];
      const uint32_t lo01 = __builtin_amdgcn_perm(d1, d0, 0x05010400u);
      const uint32_t hi01 = __builtin_amdgcn_perm(d1, d0, 0x07030602u);
      const uint32_t lo23 = __builtin_amdgcn_perm(d3, d2, 0x05010400u);
      const uint32_t hi23 = __builtin_amdgcn_perm(d3, d2, 0x07030602u);
      uint32_t o[4];
      o[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
      o[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
      o[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
      o[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
      const int64_t r = r0 + 4 * rg;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + 4 * cq + j;
        uint8_t* at = qT + c * rows + r;
        if (!EDGE || (c < cols && r + 4 <= rows)) {
          __builtin_nontemporal_store(o[j], reinterpret_cast<qt_t*>(at));
        } else if (c < cols) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (r + i < rows) at[i] = (uint8_t)(o[j] >> (8 * i));
        }
      }
    }
  }
  // per tensor: the block's amax into the slot with one atomic (a plain read first: most blocks do not raise it)
  if constexpr (!TILE) {
    if (amax_slot != nullptr) {
      const uint32_t mx = wave_max_u32(amax_acc);
      __syncthreads();
      if (lane == 0) cred[wave][0] = __uint_as_float(mx);
      __syncthreads();
      if (t == 0) {
        uint32_t bm = __float_as_uint(cred[0][0]);
#pragma unroll
        for (int w = 1; w < 8; ++w) bm = bm > __float_as_uint(cred[w][0]) ? bm : __float_as_uint(cred[w][0]);
        if (bm > __hip_atomic_load(amax_slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(amax_slot, bm);
      }
    }
  }
}

struct ActArgs {
  const void *dh, *pre;
  int64_t rows, cols;  // of the result
  const float* scale;
  float* amax;
  uint8_t* q;
  float* q_sinv;
  uint8_t* qT;
  float* qT_sinv;
  float* part;
  hipStream_t st;
};

template <int OP, int FMT, bool BF16>
static void launch_act(const ActArgs& a, bool tile) {
  const int64_t tiles = ((a.rows + kActTile - 1) / kActTile) * ((a.cols + kActTile - 1) / kActTile);
  const int64_t cap = 24ll * device_cus();
  const dim3 grid((unsigned)(tile ? tiles : std::min(tiles, cap)));
  uint32_t* slot = reinterpret_cast<uint32_t*>(a.amax);
#define SFP8_ACT(TILE, EDGE)                                                                                          \
  hipLaunchKernelGGL((act_ct_kernel<OP, FMT, BF16, TILE, EDGE>), grid, dim3(512), 0, a.st, a.dh, a.pre, a.rows, a.cols, \
                     a.scale, slot, a.q, a.q_sinv, a.qT, a.qT_sinv, a.part)
  if (tile) SFP8_ACT(true, false);
  else if (a.rows % kActTile == 0 && a.cols % kActTile == 0) SFP8_ACT(false, false);
  else SFP8_ACT(false, true);
#undef SFP8_ACT
}

template <int OP>
static void launch_act_types(const ActArgs& a, int fmt, bool bf16, bool tile) {
  if (fmt == FP8_E4M3) {
    if (bf16) launch_act<OP, FP8_E4M3, true>(a, tile);
    else launch_act<OP, FP8_E4M3, false>(a, tile);
  } else {
    if (bf16) launch_act<OP, FP8_E5M2, true>(a, tile);
    else launch_act<OP, FP8_E5M2, false>(a, tile);
  }
}

// the checks that both entry points share; H = columns of the result
static int act_check(const char* what, int dtype, int64_t rows, int64_t cols, int act, int fmt, int granularity,
                     int64_t H, const float* scale, const float* amax_slot, const float* q_sinv, const float* qT_sinv) {
  SFP8_REQUIRE(dtype == HP_F32 || dtype == HP_BF16, FP8_ERR_DTYPE, "%s: dtype %d", what, dtype);
  SFP8_REQUIRE(fmt == FP8_E4M3 || fmt == FP8_E5M2, FP8_ERR_ARG, "%s: fmt %d", what, fmt);
  SFP8_REQUIRE(granularity == FP8_SCALE_TENSOR || granularity == FP8_SCALE_TILE_1x128, FP8_ERR_ARG,
               "%s: granularity %d (TENSOR or TILE_1x128)", what, granularity);
  SFP8_REQUIRE(rows >= 0 && cols >= 0, FP8_ERR_SHAPE, "%s: negative shape", what);
  SFP8_REQUIRE(rows < (1ll << 31) && cols < (1ll << 31), FP8_ERR_SHAPE, "%s: dimension >= 2^31", what);
  SFP8_REQUIRE(act != FP8_ACT_SWIGLU || cols % 2 == 0, FP8_ERR_SHAPE,
               "%s: SwiGLU needs an even number of columns, cols=%lld", what, (long long)cols);
  SFP8_REQUIRE(((rows + 127) / 128) * ((cols + 127) / 128) < (1ll << 31), FP8_ERR_SHAPE, "%s: too many tiles", what);
  if (granularity == FP8_SCALE_TILE_1x128) {
    SFP8_REQUIRE(rows % 128 == 0 && H % 128 == 0, FP8_ERR_SHAPE,
                 "%s: TILE_1x128 needs rows=%lld and the result's columns=%lld to be multiples of 128", what,
                 (long long)rows, (long long)H);
    SFP8_REQUIRE(scale == nullptr && amax_slot == nullptr, FP8_ERR_ARG, "%s: TILE_1x128 takes no scale or amax_slot",
                 what);
    SFP8_REQUIRE(rows * cols == 0 || (q_sinv != nullptr && qT_sinv != nullptr && aligned4(q_sinv) && aligned4(qT_sinv)),
                 FP8_ERR_ARG, "%s: TILE_1x128 needs 4-byte aligned q_scale_inv and qT_scale_inv", what);
  } else {
    SFP8_REQUIRE(scale != nullptr && aligned4(scale), FP8_ERR_ARG, "%s: TENSOR needs a 4-byte aligned scale", what);
    SFP8_REQUIRE(amax_slot == nullptr || aligned4(amax_slot), FP8_ERR_ARG, "%s: misaligned amax_slot", what);
    SFP8_REQUIRE(q_sinv == nullptr && qT_sinv == nullptr, FP8_ERR_ARG, "%s: TENSOR writes no scale arrays", what);
  }
  return FP8_OK;
}

}  // namespace sfp8

using namespace sfp8;

extern "C" int fp8_act_cast_transpose(const void* pre, int dtype, int64_t rows, int64_t cols, int act, int fmt,
                                      int granularity, const float* scale, float* amax_slot, uint8_t* q,
                                      float* q_scale_inv, uint8_t* qT, float* qT_scale_inv, void* stream) {
  const char* what = "fp8_act_cast_transpose";
  SFP8_REQUIRE(act == FP8_ACT_GELU || act == FP8_ACT_SWIGLU, FP8_ERR_ARG, "%s: act %d (GELU or SWIGLU)", what, act);
  const int64_t H = act == FP8_ACT_SWIGLU ? cols / 2 : cols;
  const int rc = act_check(what, dtype, rows, cols, act, fmt, granularity, H, scale, amax_slot, q_scale_inv,
                           qT_scale_inv);
  if (rc != FP8_OK) return rc;
  if (rows == 0 || H == 0) return FP8_OK;
  SFP8_REQUIRE(pre != nullptr && q != nullptr && qT != nullptr, FP8_ERR_ARG, "%s: null pre, q or qT", what);
  SFP8_REQUIRE(aligned16(pre) && aligned16(q) && aligned16(qT), FP8_ERR_ARG, "%s: pre, q, qT must be 16-byte aligned",
               what);
  const ActArgs a = {nullptr, pre,         rows, H,            scale,   amax_slot,
                     q,       q_scale_inv, qT,   qT_scale_inv, nullptr, (hipStream_t)stream};
  const bool bf = dtype == HP_BF16, tile = granularity == FP8_SCALE_TILE_1x128;
  if (act == FP8_ACT_GELU) launch_act_types<ACT_FWD_GELU>(a, fmt, bf, tile);
  else launch_act_types<ACT_FWD_SWIGLU>(a, fmt, bf, tile);
  return check_launch(what);
}

extern "C" size_t fp8_act_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows >= (1ll << 31) || cols >= (1ll << 31)) return 0;
  const int64_t tile_rows = (rows + kActTile - 1) / kActTile;
  return tile_rows <= 1 ? 0 : (size_t)tile_rows * (size_t)cols * sizeof(float);
}

extern "C" int fp8_act_backward(const void* dh, const void* pre, int dtype, int64_t rows, int64_t cols, int act, int fmt,
                                int granularity, const float* scale, float* amax_slot, uint8_t* q, float* q_scale_inv,
                                uint8_t* qT, float* qT_scale_inv, float* dbias, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const char* what = "fp8_act_backward";
  SFP8_REQUIRE(act == FP8_ACT_NONE || act == FP8_ACT_GELU || act == FP8_ACT_SWIGLU, FP8_ERR_ARG, "%s: act %d", what,
               act);
  const int rc = act_check(what, dtype, rows, cols, act, fmt, granularity, cols, scale, amax_slot, q_scale_inv,
                           qT_scale_inv);
  if (rc != FP8_OK) return rc;
  SFP8_REQUIRE(act != FP8_ACT_NONE || pre == nullptr, FP8_ERR_ARG, "%s: FP8_ACT_NONE takes no pre", what);
  SFP8_REQUIRE(dbias == nullptr || aligned4(dbias), FP8_ERR_ARG, "%s: misaligned dbias", what);
  if (cols == 0) return FP8_OK;
  hipStream_t st = (hipStream_t)stream;
  // one tile row: its partial row is the sum itself
  const int tile_rows = (int)((rows + kActTile - 1) / kActTile);
  float* part = dbias == nullptr || tile_rows == 1 ? dbias : static_cast<float*>(workspace);
  if (rows > 0) {
    SFP8_REQUIRE(dh != nullptr && q != nullptr && qT != nullptr && (act == FP8_ACT_NONE || pre != nullptr), FP8_ERR_ARG,
                 "%s: null dh, pre, q or qT", what);
    SFP8_REQUIRE(aligned16(dh) && aligned16(pre) && aligned16(q) && aligned16(qT), FP8_ERR_ARG,
                 "%s: dh, pre, q, qT must be 16-byte aligned", what);
    const size_t need = fp8_act_backward_workspace(rows, cols);
    SFP8_REQUIRE(dbias == nullptr || need == 0 || (workspace != nullptr && aligned16(workspace) && workspace_bytes >= need),
                 FP8_ERR_ARG, "%s: dbias needs a workspace of %zu bytes, 16-byte aligned (%zu given)", what, need,
                 workspace_bytes);
    const ActArgs a = {dh, pre, rows, cols, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv, part, st};
    const bool bf = dtype == HP_BF16, tile = granularity == FP8_SCALE_TILE_1x128;
    if (act == FP8_ACT_NONE) launch_act_types<ACT_BWD_NONE>(a, fmt, bf, tile);
    else if (act == FP8_ACT_GELU) launch_act_types<ACT_BWD_GELU>(a, fmt, bf, tile);
    else launch_act_types<ACT_BWD_SWIGLU>(a, fmt, bf, tile);
    const int rc2 = check_launch(what);
    if (rc2 != FP8_OK) return rc2;
  }
  if (dbias == nullptr || tile_rows == 1) return FP8_OK;
  launch_col_reduce(part, tile_rows, 1, cols, cols, dbias, nullptr, st);
  return check_launch(what);
}
