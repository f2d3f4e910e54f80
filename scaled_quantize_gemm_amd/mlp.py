"""Python binding of the MLP block's C ABI (include/scaled_fp8_mlp.h): LayerNorm forward and backward, the
activation's cast-transpose forward and backward, and the FP8 GEMM with a residual.

Argument marshalling only, as the package's other functions; outputs and workspaces not supplied are allocated
with torch on the inputs' device.  The calls run on the tensors' device whichever device is current.
"""

from __future__ import annotations

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


_HP, _ONLY_F32, _ONLY_U8 = (_BF16, _F32), (_F32,), (_U8,)


def _arg(t: Optional[torch.Tensor], name: str, dtypes: tuple, shape: tuple) -> Optional[int]:
    """Address of an argument of one of `dtypes` and exactly `shape`, contiguous; the package's errors otherwise.  One
    test on the way of a right call: a small call's time is its marshalling."""
    if t is None:
        return None
    if not (type(t) is torch.Tensor and t.dtype in dtypes and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtypes, shape=shape)
    return t.data_ptr()


def _scalar(t: Optional[torch.Tensor], name: str) -> Optional[int]:
    """Address of an fp32 scalar (the first of at least one)."""
    if t is None:
        return None
    _need(t, name, _F32, min_numel=1)
    return t.data_ptr()


def _together(*tensors: Optional[torch.Tensor]) -> bool:
    """Whether every given tensor is on the first one's GPU."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            return False
    return dev >= 0


def _launch(t: torch.Tensor, fn, *args) -> None:
    """fn(*args, stream) on t's device and its current stream (a stream handle alone does not choose the device)."""
    if torch.cuda.current_device() == t.get_device():
        rc = fn(*args, _stream(t))
    else:
        with torch.cuda.device(t.device):
            rc = fn(*args, _stream(t))
    _check(rc)


def fp8_layernorm(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float,
                  out_dtype: Optional[int] = None, y: Optional[torch.Tensor] = None, mu: Optional[torch.Tensor] = None,
                  rsigma: Optional[torch.Tensor] = None) -> torch.Tensor:
    """LayerNorm over the last dim of x [rows][cols] -> y (OUT_F32 / OUT_BF16; by default x's type).  mu, rsigma:
    fp32 [rows] buffers for the row statistics that the backward needs."""
    _need(x, "x", _HP)
    rows, cols = _as2d(x)
    if out_dtype is None:
        out_dtype = OUT_F32 if x.dtype == _F32 else OUT_BF16
    if out_dtype not in (OUT_F32, OUT_BF16):
        raise ValueError(f"out_dtype {out_dtype}: fp8_layernorm writes OUT_F32 or OUT_BF16")
    out = _OUT_TORCH[out_dtype]
    p_gamma = _arg(gamma, "gamma", _HP, (cols,))
    p_beta = _arg(beta, "beta", (gamma.dtype,), (cols,))
    _arg(y, "y", (out,), x.shape)
    p_mu = _arg(mu, "mu", _ONLY_F32, (rows,))
    p_rs = _arg(rsigma, "rsigma", _ONLY_F32, (rows,))
    if not _together(x, gamma, beta, y, mu, rsigma):
        _on_device(x=x, gamma=gamma, beta=beta, y=y, mu=mu, rsigma=rsigma)
    if y is None:
        y = torch.empty_like(x, dtype=out)
    _launch(x, lib.fp8_layernorm, x.data_ptr(), _hp_dtype(x), rows, cols, p_gamma, p_beta, _hp_dtype(gamma), eps,
            y.data_ptr(), out_dtype, p_mu, p_rs)
    return y


def fp8_layernorm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mu: torch.Tensor,
                           rsigma: torch.Tensor, dres: Optional[torch.Tensor] = None,
                           dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                           dbeta: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of LayerNorm -> (dx [rows][cols] in x's type, dgamma [cols], dbeta [cols] in fp32); dres, of x's
    type, is added to dx.  workspace: uint8, fp8_layernorm_backward_workspace(rows, cols) bytes."""
    _need(x, "x", _HP)
    rows, cols = _as2d(x)
    shape, same = x.shape, (x.dtype,)
    p_dy = _arg(dy, "dy", _HP, shape)
    p_gamma = _arg(gamma, "gamma", _HP, (cols,))
    p_mu = _arg(mu, "mu", _ONLY_F32, (rows,))
    p_rs = _arg(rsigma, "rsigma", _ONLY_F32, (rows,))
    p_dres = _arg(dres, "dres", same, shape)
    _arg(dx, "dx", same, shape)
    _arg(dgamma, "dgamma", _ONLY_F32, (cols,))
    _arg(dbeta, "dbeta", _ONLY_F32, (cols,))
    need = lib.fp8_layernorm_backward_workspace(rows, cols)
    _need(workspace, "workspace", _U8, min_numel=need)
    if not _together(x, dy, gamma, mu, rsigma, dres, dx, dgamma, dbeta, workspace):
        _on_device(x=x, dy=dy, gamma=gamma, mu=mu, rsigma=rsigma, dres=dres, dx=dx, dgamma=dgamma, dbeta=dbeta,
                   workspace=workspace)
    if dx is None:
        dx = torch.empty_like(x)
    if dgamma is None:
        dgamma = torch.empty_like(gamma, dtype=_F32)
    if dbeta is None:
        dbeta = torch.empty_like(gamma, dtype=_F32)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=_U8, device=x.device)
    _launch(x, lib.fp8_layernorm_backward, p_dy, _hp_dtype(dy), x.data_ptr(), _hp_dtype(x), rows, cols, p_gamma,
            _hp_dtype(gamma), p_mu, p_rs, p_dres, dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(),
            _ptr(workspace), workspace.numel() if workspace is not None else 0)
    return dx, dgamma, dbeta


def _cast_outputs(rows: int, cols: int, granularity: int, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv):
    """Addresses of scale and amax_slot, and checks of the caller's outputs, for a result of [rows][cols]."""
    pointers = _scalar(scale, "scale"), _scalar(amax_slot, "amax_slot")
    _arg(q, "q", _ONLY_U8, (rows, cols))
    _arg(qT, "qT", _ONLY_U8, (cols, rows))
    if granularity != FP8_SCALE_TENSOR:
        _arg(q_scale_inv, "q_scale_inv", _ONLY_F32, (cols // 128, rows))
        _arg(qT_scale_inv, "qT_scale_inv", _ONLY_F32, (rows // 128, cols))
    return pointers


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
    _need(pre, "pre", _HP)
    rows, cols = _as2d(pre)
    width = cols // 2 if act == FP8_ACT_SWIGLU else cols
    p_scale, p_slot = _cast_outputs(rows, width, granularity, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv)
    if not _together(pre, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv):
        _on_device(pre=pre, scale=scale, amax_slot=amax_slot, q=q, q_scale_inv=q_scale_inv, qT=qT,
                   qT_scale_inv=qT_scale_inv)
    q, q_scale_inv, qT, qT_scale_inv = _new_cast_outputs(rows, width, granularity, q, q_scale_inv, qT, qT_scale_inv,
                                                         pre.device)
    _launch(pre, lib.fp8_act_cast_transpose, pre.data_ptr(), _hp_dtype(pre), rows, cols, act, fmt, granularity, p_scale,
            p_slot, q.data_ptr(), _ptr(q_scale_inv), qT.data_ptr(), _ptr(qT_scale_inv))
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
    _need(dh, "dh", _HP)
    if pre is None:
        if act != FP8_ACT_NONE:
            raise ValueError("pre is required unless act is FP8_ACT_NONE")
        rows, cols = _as2d(dh)
        p_pre = None
    else:
        _need(pre, "pre", dh.dtype)
        rows, cols = _as2d(pre)
        width = cols // 2 if act == FP8_ACT_SWIGLU else cols
        if _as2d(dh) != (rows, width):
            raise ValueError(f"dh must have shape {(rows, width)}, got {tuple(dh.shape)}")
        p_pre = pre.data_ptr()
    p_scale, p_slot = _cast_outputs(rows, cols, granularity, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv)
    _arg(dbias, "dbias", _ONLY_F32, (cols,))
    with_bias = want_dbias or dbias is not None
    need = lib.fp8_act_backward_workspace(rows, cols) if with_bias else 0
    _need(workspace, "workspace", _U8, min_numel=need)
    if not _together(dh, pre, scale, amax_slot, q, q_scale_inv, qT, qT_scale_inv, dbias, workspace):
        _on_device(dh=dh, pre=pre, scale=scale, amax_slot=amax_slot, q=q, q_scale_inv=q_scale_inv, qT=qT,
                   qT_scale_inv=qT_scale_inv, dbias=dbias, workspace=workspace)
    q, q_scale_inv, qT, qT_scale_inv = _new_cast_outputs(rows, cols, granularity, q, q_scale_inv, qT, qT_scale_inv,
                                                         dh.device)
    if with_bias:
        if dbias is None:
            dbias = torch.empty(cols, dtype=_F32, device=dh.device)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=_U8, device=dh.device)
    _launch(dh, lib.fp8_act_backward, dh.data_ptr(), p_pre, _hp_dtype(dh), rows, cols, act, fmt, granularity, p_scale,
            p_slot, q.data_ptr(), _ptr(q_scale_inv), qT.data_ptr(), _ptr(qT_scale_inv), _ptr(dbias), _ptr(workspace),
            workspace.numel() if workspace is not None else 0)
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
    out = _OUT_TORCH[out_dtype]
    p_res = _arg(residual, "residual", (out,), (M, cols))
    _arg(C, "C", (out,), (M, cols))
    p_bias = _arg(bias, "bias", _HP, (N,))
    if not _together(A, B, a_scale_inv, b_scale_inv, residual, C, bias):
        _on_device(A=A, B=B, a_scale_inv=a_scale_inv, b_scale_inv=b_scale_inv, residual=residual, C=C, bias=bias)
    if C is None:
        C = torch.empty_like(residual)
    _launch(A, lib.fp8_gemm_residual, A.data_ptr(), fmt_a, a_scale_inv.data_ptr(), gran_a, B.data_ptr(), fmt_b,
            b_scale_inv.data_ptr(), gran_b, p_bias, _hp_dtype(bias) if bias is not None else HP_F32, act, p_res,
            C.data_ptr(), out_dtype, M, N, K)
    return C


def fp8_layernorm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of fp8_layernorm_backward."""
    return lib.fp8_layernorm_backward_workspace(rows, cols)


def fp8_act_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of fp8_act_backward with dbias."""
    return lib.fp8_act_backward_workspace(rows, cols)
