"""The MLP block's operators on the CPU: the header, the exports, every refusal before a launch, and the
oracle's gradients against central differences."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import epilogue as oe, layernorm as oln, mlp as om

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "scaled_fp8_mlp.h")

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: the calls below fail validation first
OFF8 = ctypes.c_void_p(0x100008)
OFF2 = ctypes.c_void_p(0x100002)
EPS = ctypes.c_float(1e-5)


@pytest.fixture(scope="module")
def sq():
    import scaled_quantize_gemm_amd as m

    return m


def test_header_exports_and_binding_agree(sq):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(fp8_\w+)\s*\(", src, re.M)))
    assert names == sorted(sq.EXPORTED_MLP)
    for name in names:
        assert hasattr(sq.lib, name) and hasattr(sq, name), name


def test_layernorm_refusals(sq):
    f = sq.lib.fp8_layernorm

    def ln(x=FAKE, xt=1, r=4, c=768, g=FAKE, b=None, wt=1, eps=EPS, y=FAKE, yt=1, mu=None, rs=None):
        return f(x, xt, r, c, g, b, wt, eps, y, yt, mu, rs, None)

    assert ln(xt=2) == ln(wt=5) == ln(yt=2) == ln(yt=3) == sq.FP8_ERR_DTYPE
    assert ln(r=-1) == ln(c=-1) == ln(c=32769) == ln(r=1 << 31) == sq.FP8_ERR_SHAPE
    assert ln(eps=ctypes.c_float(-1)) == ln(eps=ctypes.c_float(float("nan"))) == sq.FP8_ERR_ARG
    assert ln(x=None) == ln(g=None) == ln(y=None) == sq.FP8_ERR_ARG
    assert ln(x=OFF8) == ln(y=OFF8) == ln(g=OFF8) == ln(b=OFF8) == ln(mu=OFF2) == ln(rs=OFF2) == sq.FP8_ERR_ARG
    assert ln(xt=0, yt=1) == sq.FP8_ERR_ARG  # in place with another type
    assert "one type" in sq.fp8_last_error()
    assert ln(x=None, r=0) == ln(x=None, c=0) == sq.FP8_OK


def test_layernorm_backward_refusals(sq):
    f = sq.lib.fp8_layernorm_backward
    need = sq.fp8_layernorm_backward_workspace(40, 768)
    P, Q = ctypes.c_void_p(0x200000), ctypes.c_void_p(0x300000)

    def lnb(dy=FAKE, dt=1, x=P, xt=1, r=40, c=768, g=FAKE, wt=1, mu=FAKE, rs=FAKE, dres=None, dx=Q, dg=FAKE, db=None,
            ws=FAKE, n=need):
        return f(dy, dt, x, xt, r, c, g, wt, mu, rs, dres, dx, dg, db, ws, n, None)

    assert lnb(dt=2) == lnb(xt=4) == lnb(wt=-1) == sq.FP8_ERR_DTYPE
    assert lnb(r=-1) == lnb(c=-1) == lnb(c=32769) == lnb(r=1 << 31) == sq.FP8_ERR_SHAPE
    for k in ("dy", "x", "g", "mu", "rs", "dx", "dg", "ws"):
        assert lnb(**{k: None}) == sq.FP8_ERR_ARG, k
    for k in ("dy", "x", "g", "dres", "dx", "ws"):
        assert lnb(**{k: OFF8}) == sq.FP8_ERR_ARG, k
    for k in ("mu", "rs", "dg", "db"):
        assert lnb(**{k: OFF2}) == sq.FP8_ERR_ARG, k
    assert need > 0 and lnb(n=need - 1) == sq.FP8_ERR_ARG
    assert "workspace" in sq.fp8_last_error()
    assert lnb(dx=P) == sq.FP8_ERR_ARG  # dx = x
    assert lnb(dy=Q, dt=0) == sq.FP8_ERR_ARG  # dx = dy of another type
    assert lnb(dy=None, c=0) == sq.FP8_OK
    w = sq.fp8_layernorm_backward_workspace
    assert w(4, 768) == 0  # one block
    assert w(-1, 768) == w(4, 32769) == w(1 << 31, 8) == w(4, -8) == 0


@pytest.mark.parametrize("backward", [False, True])
def test_act_refusals(sq, backward):
    need = sq.fp8_act_backward_workspace(256, 256)
    assert need > 0
    P = ctypes.c_void_p(0x200000)

    def act(dh=FAKE, pre=FAKE, dt=1, r=256, c=256, a=1, fmt=0, gran=0, s=FAKE, slot=None, q=FAKE, qs=None, qT=FAKE,
            qTs=None, db=FAKE, ws=P, n=need):
        if backward:
            return sq.lib.fp8_act_backward(dh, pre, dt, r, c, a, fmt, gran, s, slot, q, qs, qT, qTs, db, ws, n, None)
        return sq.lib.fp8_act_cast_transpose(pre, dt, r, c, a, fmt, gran, s, slot, q, qs, qT, qTs, None)

    tile = dict(gran=1, s=None, qs=FAKE, qTs=FAKE)
    assert act(dt=2) == sq.FP8_ERR_DTYPE
    assert act(a=3) == act(a=-1) == act(fmt=2) == act(gran=2) == act(gran=3) == act(gran=7) == sq.FP8_ERR_ARG
    assert act(r=-1) == act(c=-2) == act(a=2, c=255) == act(r=1 << 31) == sq.FP8_ERR_SHAPE
    assert act(**tile, r=127) == act(**tile, c=200) == sq.FP8_ERR_SHAPE
    # SwiGLU forward: the result is half as wide
    assert (act(**tile, a=2, c=128) == sq.FP8_ERR_SHAPE) == (not backward) or backward
    assert act(s=None) == act(s=OFF2) == act(slot=OFF2) == act(qs=FAKE) == act(qTs=FAKE) == sq.FP8_ERR_ARG
    assert act(**{**tile, "s": FAKE}) == act(**tile, slot=FAKE) == sq.FP8_ERR_ARG
    assert act(**{**tile, "qs": None}) == act(**{**tile, "qTs": OFF2}) == sq.FP8_ERR_ARG
    for k in ("pre", "q", "qT") + (("dh",) if backward else ()):
        assert act(**{k: None}) == sq.FP8_ERR_ARG, k
        assert act(**{k: OFF8}) == sq.FP8_ERR_ARG, k
    if backward:
        assert act(a=0) == sq.FP8_ERR_ARG  # no activation takes no pre
        assert act(db=OFF2) == act(ws=None) == act(ws=OFF8) == act(n=need - 1) == sq.FP8_ERR_ARG
        assert act(c=0) == sq.FP8_OK
        assert sq.fp8_act_backward_workspace(-1, 4) == sq.fp8_act_backward_workspace(4, -1) == 0
    else:
        assert act(a=0) == sq.FP8_ERR_ARG
        assert act(pre=None, r=0) == act(pre=None, c=0) == act(pre=None, **tile, r=0) == sq.FP8_OK


def test_gemm_residual_refusals(sq):
    def g(A=FAKE, fa=0, sa=FAKE, ga=0, B=FAKE, fb=0, sb=FAKE, gb=0, bias=None, bt=0, act=0, R=FAKE, C=FAKE, ct=1, m=4,
          n=4, k=128):
        return sq.lib.fp8_gemm_residual(A, fa, sa, ga, B, fb, sb, gb, bias, bt, act, R, C, ct, m, n, k, None)

    assert g(k=100) == g(m=-1) == g(act=2, n=5) == g(n=1 << 31) == sq.FP8_ERR_SHAPE
    assert g(ct=2) == g(ct=3) == g(ct=9) == g(bias=FAKE, bt=4) == sq.FP8_ERR_DTYPE
    assert g(fb=1) == g(fa=2) == g(act=3) == g(ga=1) == g(gb=3) == sq.FP8_ERR_ARG
    for k in ("A", "B", "R", "C"):
        assert g(**{k: None}) == g(**{k: OFF8}) == sq.FP8_ERR_ARG, k
    assert g(sa=None) == g(sb=None) == g(bias=OFF2) == sq.FP8_ERR_ARG
    assert g(A=None, R=None, m=0) == g(B=None, C=None, n=0) == sq.FP8_OK


def _raises(fn, exc, match):
    with pytest.raises(exc, match=match):
        fn()


def test_binding_rejects_mis_sized_buffers(sq):
    bf, u8 = torch.bfloat16, torch.uint8
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype)  # noqa: E731
    x, g = e(60, 40, dtype=bf), e(40)
    ln = sq.fp8_layernorm
    _raises(lambda: ln(x.half(), g, None, 1e-5), TypeError, "x must be")
    _raises(lambda: ln(x, e(39), None, 1e-5), ValueError, "gamma must have")
    _raises(lambda: ln(x, g, e(40, dtype=bf), 1e-5), TypeError, "beta must be")
    _raises(lambda: ln(x, g, None, 1e-5, sq.OUT_E4M3), ValueError, "OUT_F32 or OUT_BF16")
    _raises(lambda: ln(x, g, None, 1e-5, y=e(60, 40)), TypeError, "y must be")
    _raises(lambda: ln(x, g, None, 1e-5, mu=e(5)), ValueError, "mu must have")
    _raises(lambda: ln(e(40, 60, dtype=bf).t(), g, None, 1e-5), ValueError, "contiguous")
    _raises(lambda: ln(e(2, 3, 40), g, None, 1e-5), ValueError, "1-D or 2-D")
    _raises(lambda: ln(x, g, None, 1e-5), ValueError, "GPU tensor")
    lb = lambda **k: sq.fp8_layernorm_backward(**{**dict(dy=x, x=x, gamma=g, mu=e(60), rsigma=e(60)), **k})  # noqa: E731
    _raises(lambda: lb(dy=e(60, 39)), ValueError, "dy must have")
    _raises(lambda: lb(mu=e(60, 1)), ValueError, "mu must have")
    _raises(lambda: lb(rsigma=e(60, dtype=bf)), TypeError, "rsigma must be")
    _raises(lambda: lb(dres=e(60, 40)), TypeError, "dres must be")
    _raises(lambda: lb(dx=e(60, 41, dtype=bf)), ValueError, "dx must have")
    _raises(lambda: lb(dgamma=e(40, dtype=bf)), TypeError, "dgamma must be")
    _raises(lambda: lb(dbeta=e(41)), ValueError, "dbeta must have")
    _raises(lambda: lb(workspace=e(8, dtype=u8)), ValueError, "at least")
    _raises(lambda: lb(), ValueError, "GPU tensor")
    one, pre = e(1), e(128, 256, dtype=bf)
    ac = lambda **k: sq.fp8_act_cast_transpose(**{**dict(pre=pre, act=2, fmt=0, scale=one), **k})  # noqa: E731
    _raises(lambda: ac(q=e(128, 256, dtype=u8)), ValueError, "q must have")
    _raises(lambda: ac(qT=e(128, 128, dtype=bf)), TypeError, "qT must be")
    _raises(lambda: ac(granularity=1, scale=None, q_scale_inv=e(2, 128)), ValueError, "q_scale_inv must have")
    _raises(lambda: ac(granularity=1, scale=None, qT_scale_inv=e(1, 256)), ValueError, "qT_scale_inv must have")
    _raises(lambda: ac(scale=e(0)), ValueError, "at least 1")
    _raises(lambda: ac(), ValueError, "GPU tensor")
    pre = e(256, 256, dtype=bf)
    ab = lambda **k: sq.fp8_act_backward(  # noqa: E731
        **{**dict(dh=e(256, 128, dtype=bf), pre=pre, act=2, fmt=1, scale=one), **k})
    _raises(lambda: ab(dh=pre), ValueError, "dh must have shape")
    _raises(lambda: ab(dh=e(256, 128)), TypeError, "pre must be")
    _raises(lambda: ab(pre=None), ValueError, "pre is required")
    _raises(lambda: ab(dbias=e(128)), ValueError, "dbias must have")
    _raises(lambda: ab(qT=e(128, 256, dtype=u8)), ValueError, "qT must have")
    _raises(lambda: ab(workspace=e(4, dtype=u8)), ValueError, "at least")
    _raises(lambda: ab(), ValueError, "GPU tensor")
    A, B = e(8, 128, dtype=u8), e(16, 128, dtype=u8)
    gr = lambda R, **k: sq.fp8_gemm_residual(A, 0, one, 0, B, 0, one, 0, R, **k)  # noqa: E731
    _raises(lambda: gr(e(8, 15)), ValueError, "residual must have")
    _raises(lambda: gr(e(8, 16), out_dtype=sq.OUT_BF16), TypeError, "residual must be")
    _raises(lambda: gr(e(8, 16), act=2), ValueError, "residual must have")
    _raises(lambda: gr(e(8, 16), C=e(8, 16, dtype=bf)), TypeError, "C must be")
    _raises(lambda: gr(e(8, 16), bias=e(15)), ValueError, "bias must have")
    _raises(lambda: gr(e(8, 16), out_dtype=sq.OUT_E4M3), ValueError, "OUT_F32 or OUT_BF16")
    _raises(lambda: gr(e(8, 16)), ValueError, "GPU tensor")


def test_a_launch_makes_the_tensors_device_current(sq, monkeypatch):
    """Tensors on another device than the current one: the call runs with theirs current, on their stream."""
    import contextlib

    from scaled_quantize_gemm_amd import mlp

    class Tensor:
        device = "cuda:1"

        def get_device(self):
            return 1

    seen = []

    @contextlib.contextmanager
    def device(d):
        seen.append(("enter", d))
        yield
        seen.append(("exit", d))

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(mlp, "_stream", lambda t: 77)
    for current in (1, 0):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
        mlp._launch(Tensor(), lambda *a: seen.append(a) or 0, 5)
    assert seen == [(5, 77), ("enter", "cuda:1"), (5, 77), ("exit", "cuda:1")]
    with pytest.raises(sq.Fp8Error):
        mlp._launch(Tensor(), lambda *a: sq.FP8_ERR_ARG)


# ------------------------------------------------------------------ the oracle's gradients against differences


def _difference(f, x, h):
    """d f / d x by central differences, f a scalar of an array."""
    d = np.empty_like(x)
    for i in np.ndindex(x.shape):
        p, m = x.copy(), x.copy()
        p[i] += h
        m[i] -= h
        d[i] = (f(p) - f(m)) / (2 * h)
    return d


# the central difference of a function whose third derivative is at most D is off by h^2 D / 6, and its rounding
# by 2^-52 |f| / h: h = 1e-5 with |f|, D of order 10 gives 2e-10 and 2e-10; 1e-7 leaves room for larger D


def test_oracle_layernorm_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    x, w, gamma, beta = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), 1 + rng.standard_normal(7), rng.standard_normal(7)
    _, mean, rs = oln.layernorm_ref(x, gamma, beta, 1e-5)
    dx, dg, db = om.layernorm_backward(w, x, gamma, mean, rs)
    f = lambda x_, g_, b_: float((w * oln.layernorm_ref(x_, g_, b_, 1e-5)[0]).sum())  # noqa: E731
    assert np.abs(dx - _difference(lambda v: f(v, gamma, beta), x, 1e-5)).max() < 1e-7
    assert np.abs(dg - _difference(lambda v: f(x, v, beta), gamma, 1e-5)).max() < 1e-7
    assert np.abs(db - _difference(lambda v: f(x, gamma, v), beta, 1e-5)).max() < 1e-7
    res = rng.standard_normal((3, 7))
    assert np.array_equal(om.layernorm_backward(w, x, gamma, mean, rs, res)[0], dx + res)


@pytest.mark.parametrize("act", [oe.ACT_NONE, oe.ACT_GELU, oe.ACT_SWIGLU])
def test_oracle_activation_backward_is_the_derivative(act):
    rng = np.random.default_rng(2 + act)
    v = 2 * rng.standard_normal((4, 6))
    w = rng.standard_normal(om.activation(v, act).shape)
    d = om.activation_backward(w, v, act)
    assert np.abs(d - _difference(lambda x: float((w * om.activation(x, act)).sum()), v, 1e-5)).max() < 1e-7
