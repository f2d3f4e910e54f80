/*
 * scaled_fp8_mlp.h -- C ABI of the high-precision half of the FP8 MLP block (LayerNorm, linear +
 * activation, linear + residual) for AMD Instinct MI355X (gfx950), forward and backward.
 *
 * Beside the FP8 linear's hot path (scaled_fp8.h, same library): the steps between its GEMMs.
 * One training step of the block is
 *   forward    fp8_layernorm -> fp8_cast_transpose -> fp8_gemm_fused (activation, aux) ->
 *              fp8_act_cast_transpose (FC2's input and its transpose) -> fp8_gemm_residual
 *   backward   fp8_cast_transpose of dY -> fp8_gemm (dH) -> fp8_act_backward -> fp8_gemm dgrad and
 *              wgrad -> fp8_layernorm_backward (with the residual branch's gradient)
 *
 * Sources (web pages): Transformer Engine fused-kernels tutorial, module tour cell
 * (te.LayerNorm, te.LayerNormMLP, te.Linear(bias=True)) and plain-PyTorch block cell
 * (x + MLP(LayerNorm(x)), nn.GELU); "Week 14" course page, MoE exercise (SwiGLU) and absmax bullet
 * (1x128 runs); "Transformer Scaling" lesson, Part 01 (E4M3 forward, E5M2 gradients, delayed
 * scales).  The pages give modules, not gradients: those are the formulas below.
 *
 * The conventions, enums, error codes and fp8_last_error() of scaled_fp8.h hold: device pointers
 * owned by the caller, row-major contiguous matrices, 16-byte aligned data pointers, work enqueued
 * on `stream`, no allocation, no state.  A workspace is scratch memory of one call: its contents
 * need not be initialised and mean nothing afterwards, and calls that may run at the same time
 * (other streams, branches of a graph) need one each.
 */
#ifndef SCALED_FP8_MLP_H
#define SCALED_FP8_MLP_H

#include "scaled_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8_layernorm -- LayerNorm with a high-precision output.
 *   x          device, x_dtype HP_F32 or HP_BF16, [rows][cols]
 *   gamma      device, w_dtype HP_F32 or HP_BF16, [cols]; beta the same or NULL (no shift)
 *   eps        >= 0
 *   Per row, in fp32: mean = sum(x) / cols; var = sum((x - mean)^2) / cols;
 *   rs = 1 / sqrt(var + eps); y = (x - mean) * rs * gamma + beta.
 *   y          device, y_dtype OUT_F32 or OUT_BF16 (round to nearest even), [rows][cols]
 *   mu, rsigma device fp32 [rows] (mean and rs, for the backward), or NULL
 *   Any rows; 1 <= cols <= 32768, of any residue.  Empty inputs are a no-op.  y may be x itself
 *   where both have one type.  A row with a NaN or an infinity gives NaN throughout.
 *   Alignment: x, y, gamma, beta 16-byte; mu, rsigma 4-byte.
 *   Errors: FP8_ERR_ARG, FP8_ERR_SHAPE (negative sizes, cols > 32768, rows >= 2^31),
 *           FP8_ERR_DTYPE.
 */
int fp8_layernorm(const void *x, int x_dtype, int64_t rows, int64_t cols, const void *gamma, const void *beta,
                  int w_dtype, float eps, void *y, int y_dtype, float *mu, float *rsigma, void *stream);

/*
 * fp8_layernorm_backward -- gradients of LayerNorm, with the reductions of its weights' gradients.
 *   dy         device, dy_dtype HP_F32 or HP_BF16, [rows][cols]
 *   x, x_dtype, gamma, w_dtype: as in the forward; mu, rsigma as it wrote them (fp8_layernorm or
 *   fp8_layernorm_quantize)
 *   dres       device, of x's type, [rows][cols]: the gradient that reaches x past the norm (the
 *              residual branch), added to dx; or NULL
 *   With xh = (x - mu) * rsigma and g = dy * gamma, per row in fp32:
 *     dx = rsigma * (g - mean(g) - xh * mean(g * xh)) + dres
 *   and over the rows, in fp32: dgamma = sum dy * xh, dbeta = sum dy.
 *   dx         device, of x's type, [rows][cols]; may be dres itself, or dy itself where dy has
 *              x's type
 *   dgamma     device fp32 [cols]; dbeta the same or NULL.  Overwritten; zero for rows == 0.
 *              The order of the sums is fixed by rows, cols, the types and the device: the same
 *              call gives the same bits.
 *   workspace  device, 16-byte aligned, at least fp8_layernorm_backward_workspace(rows, cols) bytes
 *   Any rows; 1 <= cols <= 32768 (cols == 0 is a no-op).
 *   Alignment: dy, x, gamma, dres, dx 16-byte; mu, rsigma, dgamma, dbeta 4-byte.
 *   Errors: FP8_ERR_ARG (also a workspace that is too small), FP8_ERR_SHAPE, FP8_ERR_DTYPE.
 */
int fp8_layernorm_backward(const void *dy, int dy_dtype, const void *x, int x_dtype, int64_t rows, int64_t cols,
                           const void *gamma, int w_dtype, const float *mu, const float *rsigma, const void *dres,
                           void *dx, float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes,
                           void *stream);
/* Bytes of workspace for that call (0 where it needs none, and for sizes it refuses). */
size_t fp8_layernorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * fp8_act_cast_transpose -- activation of a saved pre-activation, cast to FP8 with its transpose.
 *   pre        device, dtype HP_F32 or HP_BF16, [rows][cols] (fp8_gemm_fused's aux copy is bf16)
 *   act        FP8_ACT_GELU:   h = v * Phi(v), [rows][cols]
 *              FP8_ACT_SWIGLU: h[f] = silu(v[2f]) * v[2f+1], [rows][cols/2] (cols even)
 *              (for no activation: fp8_cast_transpose, fp8_cast_transpose_blockwise)
 *   With H = cols (GELU) or cols/2 (SwiGLU) and h in fp32:
 *   granularity FP8_SCALE_TENSOR: q = enc(fp32(h * scale[0])) [rows][H], qT = q transposed [H][rows];
 *              amax_slot (may be NULL) max-reduced with max |h|; the scale arrays must be NULL.
 *              Any rows, cols.
 *              FP8_SCALE_TILE_1x128: as fp8_cast_transpose_blockwise(TILE_1x128) of h: q with one
 *              scale per 1x128 run, q_scale_inv = fp32 [H/128][rows]; qT with one per 128x1 run of
 *              h, qT_scale_inv = fp32 [rows/128][H].  rows % 128 == 0, H % 128 == 0; scale and
 *              amax_slot must be NULL.
 *   q, qT      device uint8.  Empty inputs are a no-op.  GELU of +inf is +inf, of -inf 0; elements
 *   that are not finite are cast as fp8_quantize casts them.
 *   Alignment: pre, q, qT 16-byte; fp32 scalars and arrays 4-byte.
 *   Errors: FP8_ERR_ARG, FP8_ERR_SHAPE, FP8_ERR_DTYPE.
 */
int fp8_act_cast_transpose(const void *pre, int dtype, int64_t rows, int64_t cols, int act, int fmt, int granularity,
                           const float *scale, float *amax_slot, uint8_t *q, float *q_scale_inv, uint8_t *qT,
                           float *qT_scale_inv, void *stream);

/*
 * fp8_act_backward -- gradient of the activation, cast to FP8 with its transpose, and the bias
 * gradient: from dh to what FC1's dgrad (q) and wgrad (qT) multiply.
 *   dh         device, dtype HP_F32 or HP_BF16, [rows][H] (H = cols, SwiGLU: cols/2)
 *   pre        device, of the same dtype, [rows][cols]; NULL for FP8_ACT_NONE
 *   act        FP8_ACT_NONE:   d = dh (the cast and bias gradient of a linear without activation)
 *              FP8_ACT_GELU:   d = dh * (Phi(v) + v * phi(v)), phi the normal density
 *              FP8_ACT_SWIGLU: with s = 1 / (1 + e^-g): d[2f] = dh[f] * u * s * (1 + g (1 - s)),
 *                              d[2f+1] = dh[f] * g * s  (g = v[2f], u = v[2f+1])
 *   A pre-activation that is not finite gives what fp32 arithmetic makes of these formulas (NaN for
 *   an infinity times 0); its element alone is touched, in its tile's runs scale 1.
 *   q [rows][cols], qT [cols][rows], scale, amax_slot, q_scale_inv, qT_scale_inv: d cast as
 *   fp8_act_cast_transpose casts h (the shapes with cols in place of H).
 *   dbias      device fp32 [cols]: sum over the rows of d in fp32, before the cast; or NULL.
 *              Overwritten; zero for rows == 0.  A fixed order of sums, as for dgamma above.
 *   workspace  device, 16-byte aligned, at least fp8_act_backward_workspace(rows, cols) bytes; NULL
 *              and 0 will do without dbias
 *   Errors: FP8_ERR_ARG (also a workspace that is too small), FP8_ERR_SHAPE, FP8_ERR_DTYPE.
 */
int fp8_act_backward(const void *dh, const void *pre, int dtype, int64_t rows, int64_t cols, int act, int fmt,
                     int granularity, const float *scale, float *amax_slot, uint8_t *q, float *q_scale_inv,
                     uint8_t *qT, float *qT_scale_inv, float *dbias, void *workspace, size_t workspace_bytes,
                     void *stream);
/* Bytes of workspace for that call with dbias (0 where it needs none, and for sizes it refuses). */
size_t fp8_act_backward_workspace(int64_t rows, int64_t cols);

/*
 * fp8_gemm_residual -- fp8_gemm with bias, activation and a residual in its epilogue.
 *   A, B, scales, granularities, M, N, K: as fp8_gemm_fused (B must be E4M3).
 *   Per output element, in fp32: v = the dequantised GEMM result; v = v + bias[n] if bias != NULL;
 *   y = act(v) as fp8_gemm_fused (SwiGLU: N even, N/2 columns); C = y + residual.
 *   residual, C  device, c_dtype OUT_F32 or OUT_BF16 (round to nearest even), [M][N or N/2].  C may
 *                be the residual itself (a residual stream kept in place, or a weight gradient
 *                accumulated over micro-batches); they must not overlap otherwise.
 *   Few rows (a decoding step's tokens) run on a kernel that splits K over a block's waves: the
 *   sums' order, and with it the last bits, differ from fp8_gemm's there.
 *   Alignment: C, residual 16-byte; bias as fp8_gemm_fused.
 *   Errors: as fp8_gemm_fused.
 */
int fp8_gemm_residual(const uint8_t *A, int fmt_a, const void *a_scale_inv, int gran_a, const uint8_t *B, int fmt_b,
                      const void *b_scale_inv, int gran_b, const void *bias, int bias_dtype, int act,
                      const void *residual, void *C, int c_dtype, int64_t M, int64_t N, int64_t K, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SCALED_FP8_MLP_H */
