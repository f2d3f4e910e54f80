"""Python binding of the MLP block's C ABI (include/scaled_fp8_mlp.h): LayerNorm forward and backward, the
activation's cast-transpose forward and backward, and the FP8 GEMM with a residual.

Argument marshalling only, as the package's other functions; outputs and workspaces not supplied are allocated
with torch on the inputs' device.  The calls run on the tensors' device whichever device is current.
"""

from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import (_as2d, _check, _gemm_operands, _hp_dtype, _need, _on_device, _OUT_TORCH, _ptr, _stream, FP8_ACT_NONE,
               FP8_ACT_SWIGLU, FP8_SCALE_TENSOR, HP_F32, OUT_BF16, OUT_F32, lib)

EXPORTED_MLP = ("fp8_layernorm", "fp8_layernorm_backward", "fp8_layernorm_backward_workspace",
                "fp8_act_cast_transpose", "fp8_act_backward", "fp8_act_backward_workspace", "fp8_gemm_residual")

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
lib.fp8_layernorm.argtypes = [_vp, _i32, _i64, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _i32, _vp, _vp, _vp]
lib.fp8_layernorm_backward.argtypes = [_vp, _i32, _vp, _i32, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _sz, _vp]
lib.fp8_act_cast_transpose.argtypes = [_vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.fp8_act_backward.argtypes = [_vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _sz, _vp]
lib.fp8_gemm_residual.argtypes = [_vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _i32, _i64,
                                  _i64, _i64, _vp]
for _name in ("fp8_layernorm_backward_workspace", "fp8_act_backward_workspace"):
    getattr(lib, _name).argtypes = [_i64, _i64]
    getattr(lib, _name).restype = _sz

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8


def _current(t: torch.Tensor):
    """The tensor's device made current for a launch (a stream handle alone does not choose the device)."""
    if torch.cuda.current_device() == t.device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _scratch(workspace: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    """The caller's workspace, or one of `need` bytes (on the current stream, as the call)."""
    if workspace is None:
        return torch.empty(need, dtype=_U8, device=device)
    return workspace


def fp8_layernorm(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float,
                  out_dtype: Optional[int] = None, y: Optional[torch.Tensor] = None, mu: Optional[torch.Tensor] = None,
                  rsigma: Optional[torch.Tensor] = None) -> torch.Tensor:
    """LayerNorm over the last dim of x [rows][cols] -> y (OUT_F32 / OUT_BF16; by default x's type).  mu, rsigma:
    fp32 [rows] buffers for the row statistics that the backward needs."""
    _need(x, "x", (_BF16, _F32))
    rows, cols = _as2d(x)
    if out_dtype is None:
        out_dtype = OUT_F32 if x.dtype == _F32 else OUT_BF16
    if out_dtype not in (OUT_F32, OUT_BF16):
        raise ValueError(f"out_dtype {out_dtype}: fp8_layernorm writes OUT_F32 or OUT_BF16")
    _need(gamma, "gamma", (_BF16, _F32), shape=(cols,))
    _need(beta, "beta", gamma.dtype, shape=(cols,))
    _need(y, "y", _OUT_TORCH[out_dtype], shape=tuple(x.shape))
    _need(mu, "mu", _F32, shape=(rows,))
    _need(rsigma, "rsigma", _F32, shape=(rows,))
    _on_device(x=x, gamma=gamma, beta=beta, y=y, mu=mu, rsigma=rsigma)
    if y is None:
        y = torch.empty(x.shape, dtype=_OUT_TORCH[out_dtype], device=x.device)
    with _current(x):
        _check(lib.fp8_layernorm(_ptr(x), _hp_dtype(x), rows, cols, _ptr(gamma), _ptr(beta), _hp_dtype(gamma),
                                 float(eps), _ptr(y), out_dtype, _ptr(mu), _ptr(rsigma), _stream(x)))
    return y


def fp8_layernorm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mu: torch.Tensor,
                           rsigma: torch.Tensor, dres: Optional[torch.Tensor] = None,
                           dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                           dbeta: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of LayerNorm -> (dx [rows][cols] in x's type, dgamma [cols], dbeta [cols] in fp32); dres, of x's
    type, is added to dx.  workspace: uint8, fp8_layernorm_backward_workspace(rows, cols) bytes."""
    _need(x, "x", (_BF16, _F32))
    rows, cols = _as2d(x)
    shape = tuple(x.shape)
    _need(dy, "dy", (_BF16, _F32), shape=shape)
    _need(gamma, "gamma", (_BF16, _F32), shape=(cols,))
    _need(mu, "mu", _F32, shape=(rows,))
    _need(rsigma, "rsigma", _F32, shape=(rows,))
    _need(dres, "dres", x.dtype, shape=shape)
    _need(dx, "dx", x.dtype, shape=shape)
    _need(dgamma, "dgamma", _F32, shape=(cols,))
    _need(dbeta, "dbeta", _F32, shape=(cols,))
    need = lib.fp8_layernorm_backward_workspace(rows, cols)
    _need(workspace, "workspace", _U8, min_numel=need)
    _on_device(x=x, dy=dy, gamma=gamma, mu=mu, rsigma=rsigma, dres=dres, dx=dx, dgamma=dgamma, dbeta=dbeta,
               workspace=workspace)
    with _current(x):
        if dx is None:
            dx = torch.empty_like(x)
        if dgamma is None:
            dgamma = torch.empty(cols, dtype=_F32, device=x.device)
        if dbeta is None:
            dbeta = torch.empty(cols, dtype=_F32, device=x.device)
        ws = _scratch(workspace, need, x.device)
        _check(lib.fp8_layernorm_backward(_ptr(dy), _hp_dtype(dy), _ptr(x), _hp_dtype(x), rows, cols, _ptr(gamma),
                                          _hp_dtype(gamma), _ptr(mu), _ptr(rsigma), _ptr(dres), _ptr(dx), _ptr(dgamma),
                                          _ptr(dbeta), _ptr(ws), ws.numel(), _stream(x)))
    return dx, dgamma, dbeta


def _cast_outputs(rows: int, cols: int, granularity: int, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv) -> None:
    """Checks of the caller's cast arguments for a result of [rows][cols]."""
    _need(scale, "scale", _F32, min_numel=1)
    _need(amax_slot, "amax_slot", _F32, min_numel=1)
    _need(q, "q", _U8, shape=(rows, cols))
    _need(qT, "qT", _U8, shape=(cols, rows))
    if granularity != FP8_SCALE_TENSOR:
        _need(q_scale_inv, "q_scale_inv", _F32, shape=(cols // 128, rows))
        _need(qT_scale_inv, "qT_scale_inv", _F32, shape=(rows // 128, cols))


def _new_cast_outputs(rows: int, cols: int, granularity: int, q, q_scale_inv, qT, qT_scale_inv, device):
    if q is None:
        q = torch.empty((rows, cols), dtype=_U8, device=device)
    if qT is None:
        qT = torch.empty((cols, rows), dtype=_U8, device=device)
    if granularity != FP8_SCALE_TENSOR:
        if q_scale_inv is None:
            q_scale_inv = torch.empty((cols // 128, rows), dtype=_F32, device=device)
        if qT_scale_inv is None:
            qT_scale_inv = torch.empty((rows // 128, cols), dtype=_F32, device=device)
    return q, q_scale_inv, qT, qT_scale_inv


def fp8_act_cast_transpose(pre: torch.Tensor, act: int, fmt: int, granularity: int = FP8_SCALE_TENSOR,
                           scale: Optional[torch.Tensor] = None, amax_slot: Optional[torch.Tensor] = None,
                           q: Optional[torch.Tensor] = None, q_scale_inv: Optional[torch.Tensor] = None,
                           qT: Optional[torch.Tensor] = None, qT_scale_inv: Optional[torch.Tensor] = None):
    """GELU / SwiGLU of pre [rows][cols] cast to FP8 with its transpose -> (q [rows][H], q_scale_inv, qT [H][rows],
    qT_scale_inv), H = cols (SwiGLU: cols / 2).  TENSOR: under `scale`, amax into amax_slot, the scale arrays None;
    TILE_1x128: q_scale_inv [H/128][rows], qT_scale_inv [rows/128][H]."""
    _need(pre, "pre", (_BF16, _F32))
    rows, cols = _as2d(pre)
    width = cols // 2 if act == FP8_ACT_SWIGLU else cols
    _cast_outputs(rows, width, granularity, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv)
    _on_device(pre=pre, scale=scale, amax_slot=amax_slot, q=q, q_scale_inv=q_scale_inv, qT=qT,
               qT_scale_inv=qT_scale_inv)
    with _current(pre):
        q, q_scale_inv, qT, qT_scale_inv = _new_cast_outputs(rows, width, granularity, q, q_scale_inv, qT,
                                                             qT_scale_inv, pre.device)
        _check(lib.fp8_act_cast_transpose(_ptr(pre), _hp_dtype(pre), rows, cols, act, fmt, granularity, _ptr(scale),
                                          _ptr(amax_slot), _ptr(q), _ptr(q_scale_inv), _ptr(qT), _ptr(qT_scale_inv),
                                          _stream(pre)))
    return q, q_scale_inv, qT, qT_scale_inv


def fp8_act_backward(dh: torch.Tensor, pre: Optional[torch.Tensor], act: int, fmt: int,
                     granularity: int = FP8_SCALE_TENSOR, scale: Optional[torch.Tensor] = None,
                     amax_slot: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                     q_scale_inv: Optional[torch.Tensor] = None, qT: Optional[torch.Tensor] = None,
                     qT_scale_inv: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                     want_dbias: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradient of the activation from dh [rows][H] at pre [rows][cols] (None for FP8_ACT_NONE), cast to FP8 with its
    transpose -> (q [rows][cols], q_scale_inv, qT [cols][rows], qT_scale_inv, dbias [cols] fp32 or None).  Scaling
    as fp8_act_cast_transpose.  workspace: uint8, fp8_act_backward_workspace(rows, cols) bytes."""
    _need(dh, "dh", (_BF16, _F32))
    if pre is None:
        if act != FP8_ACT_NONE:
            raise ValueError("pre is required unless act is FP8_ACT_NONE")
        rows, cols = _as2d(dh)
    else:
        _need(pre, "pre", dh.dtype)
        rows, cols = _as2d(pre)
        width = cols // 2 if act == FP8_ACT_SWIGLU else cols
        if _as2d(dh) != (rows, width):
            raise ValueError(f"dh must have shape {(rows, width)}, got {tuple(dh.shape)}")
    _cast_outputs(rows, cols, granularity, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv)
    _need(dbias, "dbias", _F32, shape=(cols,))
    with_bias = want_dbias or dbias is not None
    need = lib.fp8_act_backward_workspace(rows, cols) if with_bias else 0
    _need(workspace, "workspace", _U8, min_numel=need)
    _on_device(dh=dh, pre=pre, scale=scale, amax_slot=amax_slot, q=q, q_scale_inv=q_scale_inv, qT=qT,
               qT_scale_inv=qT_scale_inv, dbias=dbias, workspace=workspace)
    with _current(dh):
        q, q_scale_inv, qT, qT_scale_inv = _new_cast_outputs(rows, cols, granularity, q, q_scale_inv, qT, qT_scale_inv,
                                                             dh.device)
        ws = None
        if with_bias:
            if dbias is None:
                dbias = torch.empty(cols, dtype=_F32, device=dh.device)
            ws = _scratch(workspace, need, dh.device)
        _check(lib.fp8_act_backward(_ptr(dh), _ptr(pre), _hp_dtype(dh), rows, cols, act, fmt, granularity, _ptr(scale),
                                    _ptr(amax_slot), _ptr(q), _ptr(q_scale_inv), _ptr(qT), _ptr(qT_scale_inv),
                                    _ptr(dbias), _ptr(ws), ws.numel() if ws is not None else 0, _stream(dh)))
    return q, q_scale_inv, qT, qT_scale_inv, dbias


def fp8_gemm_residual(A: torch.Tensor, fmt_a: int, a_scale_inv: torch.Tensor, gran_a: int, B: torch.Tensor, fmt_b: int,
                      b_scale_inv: torch.Tensor, gran_b: int, residual: torch.Tensor, out_dtype: Optional[int] = None,
                      bias: Optional[torch.Tensor] = None, act: int = FP8_ACT_NONE,
                      C: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = act(deq(A) . deq(B)^T + bias) + residual, fp32 or bf16 as the residual; C may be the residual."""
    M, N, K = _gemm_operands(A, a_scale_inv, gran_a, B, b_scale_inv, gran_b)
    cols = N // 2 if act == FP8_ACT_SWIGLU else N
    if out_dtype is None:
        out_dtype = OUT_F32 if residual.dtype == _F32 else OUT_BF16
    if out_dtype not in (OUT_F32, OUT_BF16):
        raise ValueError(f"out_dtype {out_dtype}: fp8_gemm_residual writes OUT_F32 or OUT_BF16")
    _need(residual, "residual", _OUT_TORCH[out_dtype], shape=(M, cols))
    _need(C, "C", _OUT_TORCH[out_dtype], shape=(M, cols))
    _need(bias, "bias", (_F32, _BF16), shape=(N,))
    _on_device(A=A, B=B, a_scale_inv=a_scale_inv, b_scale_inv=b_scale_inv, residual=residual, C=C, bias=bias)
    with _current(A):
        if C is None:
            C = torch.empty((M, cols), dtype=_OUT_TORCH[out_dtype], device=A.device)
        _check(lib.fp8_gemm_residual(_ptr(A), fmt_a, _ptr(a_scale_inv), gran_a, _ptr(B), fmt_b, _ptr(b_scale_inv),
                                     gran_b, _ptr(bias), _hp_dtype(bias) if bias is not None else HP_F32, act,
                                     _ptr(residual), _ptr(C), out_dtype, M, N, K, _stream(A)))
    return C


def fp8_layernorm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of fp8_layernorm_backward."""
    return lib.fp8_layernorm_backward_workspace(rows, cols)


def fp8_act_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of fp8_act_backward with dbias."""
    return lib.fp8_act_backward_workspace(rows, cols)
