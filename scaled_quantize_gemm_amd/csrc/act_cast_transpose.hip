// Activation (forward) and activation gradient (backward), cast to FP8 with the transpose and, backward,
// the bias gradient.
//
// forward   h = gelu(v) or silu(v[2f]) v[2f+1]
// backward  d = dh act'(v): GELU dh (Phi(v) + v phi(v)); SwiGLU (interleaved columns, s = sigmoid(g))
//           d[2f] = dh u s (1 + g (1 - s)), d[2f+1] = dh g s;  dbias = sum_rows d
// and the result goes to FP8 under the cast rules of quantize.hip, per tensor (delayed scale, amax into a
// slot) or in 1x128 runs (its own for q and for the transposed copy).
//
// One block per 128 x 128 tile of the result, which it computes into LDS in fp32 and reads by rows for q and
// by columns for qT.
#include "act_math.h"
#include "col_reduce.h"

namespace sfp8 {

constexpr int kActTile = 128, kActPitch = 129;
// what a kernel computes from its inputs
enum { ACT_FWD_GELU = 0, ACT_FWD_SWIGLU = 1, ACT_BWD_NONE = 2, ACT_BWD_GELU = 3, ACT_BWD_SWIGLU = 4 };

template <bool BF16>
__device__ __forceinline__ float act_ld(const void* __restrict__ p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}

// element (r, c) of the result [rows][cols]
template <int OP, bool BF16>
__device__ __forceinline__ float act_at(const void* __restrict__ dh, const void* __restrict__ pre, int64_t r, int64_t c,
                                        int64_t cols) {
  if constexpr (OP == ACT_FWD_GELU) return act_gelu(act_ld<BF16>(pre, r * cols + c));
  if constexpr (OP == ACT_FWD_SWIGLU)
    return act_swiglu(act_ld<BF16>(pre, 2 * (r * cols + c)), act_ld<BF16>(pre, 2 * (r * cols + c) + 1));
  if constexpr (OP == ACT_BWD_NONE) return act_ld<BF16>(dh, r * cols + c);
  if constexpr (OP == ACT_BWD_GELU) return act_ld<BF16>(dh, r * cols + c) * act_gelu_grad(act_ld<BF16>(pre, r * cols + c));
  if constexpr (OP == ACT_BWD_SWIGLU) {
    const int64_t f = r * (cols >> 1) + (c >> 1);
    float dg, du;
    act_swiglu_grad(act_ld<BF16>(dh, f), act_ld<BF16>(pre, 2 * f), act_ld<BF16>(pre, 2 * f + 1), dg, du);
    return (c & 1) ? du : dg;
  }
}

template <int FMT>
__device__ __forceinline__ uint8_t act_code(float v, float s) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return (uint8_t)nan_code(b);
  return (uint8_t)cvt_pair<FMT, false>(v * s, 0.0f, 0u);
}

template <int OP, int FMT, bool BF16, bool TILE>
__global__ void __launch_bounds__(256) act_ct_kernel(const void* __restrict__ dh, const void* __restrict__ pre,
                                                     int64_t rows, int64_t cols, const float* __restrict__ scale_p,
                                                     uint32_t* __restrict__ amax_slot, uint8_t* __restrict__ q,
                                                     float* __restrict__ q_sinv, uint8_t* __restrict__ qT,
                                                     float* __restrict__ qT_sinv, float* __restrict__ part) {
  __shared__ float v[kActTile * kActPitch];
  __shared__ float srow[kActTile], scol[kActTile];
  __shared__ uint32_t red[4];
  const int t = threadIdx.x;
  const int64_t tiles_c = (cols + kActTile - 1) / kActTile;
  const int64_t rb = blockIdx.x / tiles_c, kb = blockIdx.x % tiles_c;
  const int64_t r0 = rb * kActTile, c0 = kb * kActTile;
  uint32_t mx = 0;
  for (int e = t; e < kActTile * kActTile; e += 256) {
    const int r = e >> 7, c = e & 127;
    float x = 0.0f;
    if (r0 + r < rows && c0 + c < cols) x = act_at<OP, BF16>(dh, pre, r0 + r, c0 + c, cols);
    v[r * kActPitch + c] = x;
    mx = mx > abs_bits(x) ? mx : abs_bits(x);
  }
  __syncthreads();
  if constexpr (TILE) {
    uint32_t a = 0;
    for (int i = 0; i < kActTile; ++i) {
      const uint32_t b = abs_bits(t < 128 ? v[t * kActPitch + i] : v[i * kActPitch + t - 128]);
      a = a > b ? a : b;
    }
    float s, si;
    current_scale<FMT>(a, s, si);
    if (t < 128) {
      srow[t] = s;
      q_sinv[kb * rows + r0 + t] = si;
    } else {
      scol[t - 128] = s;
      qT_sinv[rb * cols + c0 + t - 128] = si;
    }
  } else {
    if (t < 128) srow[t] = scol[t] = *scale_p;
    mx = wave_max_u32(mx);
    if ((t & 63) == 0) red[t >> 6] = mx;
  }
  __syncthreads();
  if constexpr (!TILE) {
    if (t == 0 && amax_slot != nullptr) {
      uint32_t b = red[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) b = b > red[i] ? b : red[i];
      if (b > __hip_atomic_load(amax_slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(amax_slot, b);
    }
  }
  if (part != nullptr && t < 128 && c0 + t < cols) {
    float s = 0.0f;
    for (int r = 0; r < kActTile; ++r) s += v[r * kActPitch + t];
    part[rb * cols + c0 + t] = s;
  }
  for (int e = t; e < kActTile * kActTile; e += 256) {
    const int i = e >> 7, j = e & 127;
    if (r0 + i < rows && c0 + j < cols) q[(r0 + i) * cols + c0 + j] = act_code<FMT>(v[i * kActPitch + j], srow[i]);
    if (r0 + j < rows && c0 + i < cols) qT[(c0 + i) * rows + r0 + j] = act_code<FMT>(v[j * kActPitch + i], scol[i]);
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
  const int64_t blocks = ((a.rows + kActTile - 1) / kActTile) * ((a.cols + kActTile - 1) / kActTile);
  if (tile)
    hipLaunchKernelGGL((act_ct_kernel<OP, FMT, BF16, true>), dim3((unsigned)blocks), dim3(256), 0, a.st, a.dh, a.pre,
                       a.rows, a.cols, a.scale, reinterpret_cast<uint32_t*>(a.amax), a.q, a.q_sinv, a.qT, a.qT_sinv,
                       a.part);
  else
    hipLaunchKernelGGL((act_ct_kernel<OP, FMT, BF16, false>), dim3((unsigned)blocks), dim3(256), 0, a.st, a.dh, a.pre,
                       a.rows, a.cols, a.scale, reinterpret_cast<uint32_t*>(a.amax), a.q, a.q_sinv, a.qT, a.qT_sinv,
                       a.part);
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
  return (size_t)((rows + kActTile - 1) / kActTile) * (size_t)cols * sizeof(float);
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
  float* part = dbias != nullptr ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    SFP8_REQUIRE(dh != nullptr && q != nullptr && qT != nullptr && (act == FP8_ACT_NONE || pre != nullptr), FP8_ERR_ARG,
                 "%s: null dh, pre, q or qT", what);
    SFP8_REQUIRE(aligned16(dh) && aligned16(pre) && aligned16(q) && aligned16(qT), FP8_ERR_ARG,
                 "%s: dh, pre, q, qT must be 16-byte aligned", what);
    const size_t need = fp8_act_backward_workspace(rows, cols);
    SFP8_REQUIRE(dbias == nullptr || (workspace != nullptr && aligned16(workspace) && workspace_bytes >= need),
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
  if (dbias == nullptr) return FP8_OK;
  launch_col_reduce(part, (int)((rows + kActTile - 1) / kActTile), 1, cols, cols, dbias, nullptr, st);
  return check_launch(what);
}
