"""GPU parity of fp8_layernorm and fp8_layernorm_backward against float64.

Bounds, with u = 2^-24.  Forward: test_gpu_layernorm.ln_bound (its row sums are longer than these kernels').
Backward, at the given fp32 mu and rs: xh = (x - mu) rs takes two roundings, g = dy gamma one, g xh two more; a
row's sums, at most cols/64 sequential additions and 16 levels, round by c = (cols/64 + 16) u of their terms'
magnitudes; then the two products, two subtractions, the product with rs and the residual add.  A column's sums
add at most rows terms one after another, and not more than rows/4 + 64 where rows are shared out.  A bf16 output
is off by half a step more, 2^-8 of the value.  All are first-order sums, doubled."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from gpu_util import DEV, announce, np_of  # noqa: E402
from oracle import mlp as om  # noqa: E402
from test_gpu_layernorm import EPS, U, ln_bound  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
HALF_BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def sq():
    import scaled_quantize_gemm_amd as m

    return m


def _rand(rng, shape, std=1.0, offset=0.0, dtype=F32):
    return torch.from_numpy((std * rng.standard_normal(shape) + offset).astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check_forward(sq, rng, R, C, xt, yt, wt=F32, beta=True, offset=0.0, stats=True):
    announce("fp8_layernorm", R, C, xt, yt, wt, beta, offset)
    x, g = _rand(rng, (R, C), 1.0, offset, xt), _rand(rng, C, 0.1, 1.0, wt)
    b = _rand(rng, C, 0.1, 0.0, wt) if beta else None
    out = sq.OUT_F32 if yt == F32 else sq.OUT_BF16
    mu, rs = (torch.empty(R, device=DEV), torch.empty(R, device=DEV)) if stats else (None, None)
    y = sq.fp8_layernorm(x.to(DEV), g.to(DEV), b if b is None else b.to(DEV), EPS, out, mu=mu, rsigma=rs)
    torch.cuda.synchronize()
    assert y.dtype == yt and y.shape == (R, C)
    want, mean, rsig, e, e_mean, rel = ln_bound(f64(x), f64(g), None if b is None else f64(b), EPS)
    if yt == BF:
        e = e + HALF_BF16 * (np.abs(want) + e)
    err = np.abs(f64(y) - want)
    assert (err <= e).all(), (err - e).max()
    if stats:
        assert (np.abs(f64(mu) - mean) <= e_mean).all() and (np.abs(f64(rs) - rsig) <= rel * rsig).all()


def check_backward(sq, rng, R, C, xt, dt, wt=F32, dres=True, offset=0.0, **buffers):
    announce("fp8_layernorm_backward", R, C, xt, dt, wt, dres, offset)
    x, g = _rand(rng, (R, C), 1.0, offset, xt), _rand(rng, C, 0.1, 1.0, wt)
    dy, res = _rand(rng, (R, C), 0.01, 0.001, dt), _rand(rng, (R, C), 0.01, 0.0, xt) if dres else None
    xd = f64(x)
    mu = torch.from_numpy(xd.mean(axis=1).astype(np.float32))
    rs = torch.from_numpy((1 / np.sqrt(xd.var(axis=1) + EPS)).astype(np.float32))
    dx, dgamma, dbeta = sq.fp8_layernorm_backward(dy.to(DEV), x.to(DEV), g.to(DEV), mu.to(DEV), rs.to(DEV),
                                                  dres=None if res is None else res.to(DEV), **buffers)
    torch.cuda.synchronize()
    assert dx.dtype == xt and dgamma.dtype == dbeta.dtype == F32
    verify_backward(dx, dgamma, dbeta, dy, x, g, mu, rs, res)


def verify_backward(dx, dgamma, dbeta, dy, x, g, mu, rs, res):
    R, C = x.shape
    D, X, G, M, S = f64(dy), f64(x), f64(g), f64(mu)[:, None], f64(rs)[:, None]
    want, wg, wb = om.layernorm_backward(D, X, G, M[:, 0], S[:, 0], None if res is None else f64(res))
    xh = (X - M) * S
    gg = D * G
    c = (C / 64 + 16) * U
    m1, m2 = np.abs(gg).mean(axis=1, keepdims=True), np.abs(gg * xh).mean(axis=1, keepdims=True)
    e1, e2 = (c + 2 * U) * m1, (c + 6 * U) * m2
    e = S * (e1 + np.abs(xh) * e2 + 6 * U * (np.abs(gg) + m1 + np.abs(xh) * m2))
    e = 2 * (e + U * np.abs(want))
    if dx.dtype == BF:
        e = e + HALF_BF16 * (np.abs(want) + e)
    err = np.abs(f64(dx) - want)
    assert (err <= e).all(), ("dx", (err - e).max())
    n = min(R, R / 4 + 64)
    err, e = np.abs(f64(dgamma) - wg), 2 * (n + 5) * U * np.abs(D * xh).sum(axis=0)
    assert (err <= e).all(), ("dgamma", (err - e).max())
    err, e = np.abs(f64(dbeta) - wb), 2 * (n + 1) * U * np.abs(D).sum(axis=0)
    assert (err <= e).all(), ("dbeta", (err - e).max())


# one element, one row, fewer columns than a vector or a wave, odd widths, the edges of the register
# layouts (512 .. 32768) and just beside them
SHAPES = [(1, 1), (1, 768), (3, 7), (5, 64), (2, 8), (67, 100), (9, 513), (17, 1024), (6, 1251), (33, 2048), (7, 2056),
          (4, 4096), (5, 4104), (3, 8192), (2, 8200), (3, 10001), (2, 16384), (2, 32760), (1, 32768), (2, 32767)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
def test_forward_shapes(sq, shape, xt, yt):
    rng = np.random.default_rng(shape[0] + 5 * shape[1])
    check_forward(sq, rng, *shape, xt, yt, wt=BF if shape[1] % 3 == 0 else F32, beta=shape[0] % 2 == 1)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("xt,dt", [(BF, BF), (F32, BF), (F32, F32), (BF, F32)])
def test_backward_shapes(sq, shape, xt, dt):
    rng = np.random.default_rng(shape[0] + 7 * shape[1])
    check_backward(sq, rng, *shape, xt, dt, wt=BF if shape[1] % 3 == 0 else F32, dres=shape[0] % 2 == 1)


# few rows and many: one block, fewer rows than blocks, several rows per wave, a ragged last round
@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 9, 15, 16, 17, 32, 33, 63, 129, 300, 1023, 2051, 5000])
@pytest.mark.parametrize("cols", [96, 771, 2304])
def test_backward_row_counts(sq, rows, cols):
    check_backward(sq, np.random.default_rng(rows + cols), rows, cols, BF, BF, dres=rows % 2 == 0)


def test_large_and_offset_rows(sq):
    rng = np.random.default_rng(4)
    check_forward(sq, rng, 1500, 2048, BF, BF, wt=BF)
    check_forward(sq, rng, 64, 1024, F32, F32, offset=100.0, beta=False, stats=False)
    check_backward(sq, rng, 3000, 2048, BF, BF, wt=BF)
    check_backward(sq, rng, 64, 1024, F32, F32, offset=100.0)


def test_workload2_width_through_both(sq):
    """The norm in front of the MiniGPT layer set (2048 tokens of width 768): the backward at the statistics that the
    forward wrote."""
    rng = np.random.default_rng(8)
    x, g, dy = _rand(rng, (2048, 768), dtype=BF), _rand(rng, 768, 0.1, 1.0), _rand(rng, (2048, 768), 1e-3, dtype=BF)
    mu, rs = torch.empty(2048, device=DEV), torch.empty(2048, device=DEV)
    sq.fp8_layernorm(x.to(DEV), g.to(DEV), None, EPS, mu=mu, rsigma=rs)
    dx, dg, db = sq.fp8_layernorm_backward(dy.to(DEV), x.to(DEV), g.to(DEV), mu, rs)
    torch.cuda.synchronize()
    verify_backward(dx, dg, db, dy, x, g, mu, rs, None)


def test_same_statistics_as_the_cast_norm(sq):
    """fp8_layernorm_quantize's mu and rsigma serve the backward: within the forward's bounds of each other."""
    rng = np.random.default_rng(5)
    x, g = _rand(rng, (300, 768), dtype=BF).to(DEV), _rand(rng, 768, 0.1, 1.0).to(DEV)
    m1, r1, m2, r2 = torch.empty(4, 300, device=DEV).unbind(0)
    sq.fp8_layernorm(x, g, None, EPS, mu=m1, rsigma=r1)
    sq.fp8_layernorm_quantize(x, g, None, EPS, 0, sq.FP8_SCALE_TENSOR, scale=torch.ones(1, device=DEV), mu=m2, rsigma=r2)
    torch.cuda.synchronize()
    _, _, rs, _, e_mean, rel = ln_bound(f64(x), f64(g), None, EPS)
    assert (np.abs(f64(m1) - f64(m2)) <= 2 * e_mean).all() and (np.abs(f64(r1) - f64(r2)) <= 2 * rel * rs).all()


def test_in_place(sq):
    rng = np.random.default_rng(6)
    for C in (771, 1024):
        x, g = _rand(rng, (40, C), dtype=BF).to(DEV), _rand(rng, C, 0.1, 1.0).to(DEV)
        want = sq.fp8_layernorm(x, g, None, EPS)
        buf = x.clone()
        sq.fp8_layernorm(buf, g, None, EPS, y=buf)
        assert torch.equal(buf, want)
        dy, res = _rand(rng, (40, C), dtype=BF).to(DEV), _rand(rng, (40, C), dtype=BF).to(DEV)
        mu, rs = x.float().mean(1), 1 / x.float().std(1)
        ref = sq.fp8_layernorm_backward(dy, x, g, mu, rs, dres=res)
        for alias in ("dy", "dres"):
            a = dict(dy=dy.clone(), dres=res.clone())
            got = sq.fp8_layernorm_backward(a["dy"], x, g, mu, rs, dres=a["dres"], dx=a[alias])
            assert got[0].data_ptr() == a[alias].data_ptr()
            for p, q in zip(got, ref):
                assert torch.equal(p, q)


def test_empty(sq):
    g = torch.ones(96, device=DEV)
    none, stat = torch.empty((0, 96), device=DEV), torch.empty(0, device=DEV)
    assert sq.fp8_layernorm(none, g, None, EPS).shape == (0, 96)
    dg, db = torch.full((96,), 7.0, device=DEV), torch.full((96,), 7.0, device=DEV)
    dx, _, _ = sq.fp8_layernorm_backward(none, none, g, stat, stat, dgamma=dg, dbeta=db)
    assert dx.shape == (0, 96) and not dg.any() and not db.any()
    thin = torch.empty((4, 0), device=DEV)
    gone = torch.empty(0, device=DEV)
    assert sq.fp8_layernorm(thin, gone, None, EPS).shape == (4, 0)
    assert sq.fp8_layernorm_backward(thin, thin, gone, torch.zeros(4, device=DEV), torch.ones(4, device=DEV))[1].numel() == 0


def test_constant_and_non_finite_rows(sq):
    """A constant row gives beta exactly; a row with a NaN or an infinity gives NaN throughout and leaves the other
    rows as they are."""
    for C in (200, 771):
        x = torch.full((5, C), 3.0)
        x[1] = torch.from_numpy(np.random.default_rng(1).standard_normal(C).astype(np.float32))
        clean = x.clone()
        x[2, C // 2], x[3, 0], x[4, C - 1] = float("nan"), float("inf"), -float("inf")
        g, b = torch.full((C,), 2.0), torch.linspace(-3, 3, C)
        y = sq.fp8_layernorm(x.to(DEV), g.to(DEV), b.to(DEV), EPS).cpu()
        want = sq.fp8_layernorm(clean.to(DEV), g.to(DEV), b.to(DEV), EPS).cpu()
        assert torch.equal(y[0], b) and torch.equal(y[1], want[1]) and y[2:].isnan().all()


def test_other_stream_and_caller_buffers(sq):
    """Buffers of the caller on a stream of its own; neighbours of the outputs stay as they were."""
    rng = np.random.default_rng(9)
    for R, C in ((130, 771), (9, 771), (3, 4100)):
        _check_room(sq, rng, R, C)


def _check_room(sq, rng, R, C):
    x, g, dy = _rand(rng, (R, C)).to(DEV), _rand(rng, C, 0.1, 1.0).to(DEV), _rand(rng, (R, C)).to(DEV)
    mu, rs = x.mean(1), 1 / x.std(1)
    ref = sq.fp8_layernorm_backward(dy, x, g, mu, rs)
    torch.cuda.synchronize()
    room = torch.full((R * C + 64,), 5.0, device=DEV)
    sums = torch.full((2, C + 9), 5.0, device=DEV)
    ws = torch.full((sq.fp8_layernorm_backward_workspace(R, C) + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sq.fp8_layernorm_backward(dy, x, g, mu, rs, dx=room[:R * C].view(R, C), dgamma=sums[0, :C], dbeta=sums[1, :C],
                                  workspace=ws[:-64])
    st.synchronize()
    assert torch.equal(room[:R * C].view(R, C), ref[0]) and (room[R * C:] == 5).all()
    assert torch.equal(sums[0, :C], ref[1]) and torch.equal(sums[1, :C], ref[2]) and (sums[:, C:] == 5).all()
    assert (ws[-64:] == 0xFF).all()


def test_dbeta_may_be_left_out(sq):
    rng = np.random.default_rng(10)
    x, g, dy = _rand(rng, (50, 96)).to(DEV), _rand(rng, 96, 0.1, 1.0).to(DEV), _rand(rng, (50, 96)).to(DEV)
    mu, rs = x.mean(1), 1 / x.std(1)
    ref = sq.fp8_layernorm_backward(dy, x, g, mu, rs)
    dx, dg = torch.empty_like(x), torch.empty(96, device=DEV)
    n = sq.fp8_layernorm_backward_workspace(50, 96)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    rc = sq.lib.fp8_layernorm_backward(dy.data_ptr(), 0, x.data_ptr(), 0, 50, 96, g.data_ptr(), 0, mu.data_ptr(),
                                       rs.data_ptr(), None, dx.data_ptr(), dg.data_ptr(), None, ws.data_ptr(), n, None)
    torch.cuda.synchronize()
    assert rc == sq.FP8_OK and torch.equal(dx, ref[0]) and torch.equal(dg, ref[1])


def test_one_row_given_as_a_vector(sq):
    rng = np.random.default_rng(11)
    x, g, dy = _rand(rng, 300, dtype=BF).to(DEV), _rand(rng, 300, 0.1, 1.0).to(DEV), _rand(rng, 300, dtype=BF).to(DEV)
    mu, rs = torch.empty(2, 1, device=DEV).unbind(0)
    y = sq.fp8_layernorm(x, g, None, EPS, mu=mu, rsigma=rs)
    assert y.shape == (300,) and torch.equal(y, sq.fp8_layernorm(x[None], g, None, EPS)[0])
    dx, dg, db = sq.fp8_layernorm_backward(dy, x, g, mu, rs)
    ref = sq.fp8_layernorm_backward(dy[None], x[None], g, mu, rs)
    assert dx.shape == (300,) and torch.equal(dx, ref[0][0]) and torch.equal(dg, ref[1]) and torch.equal(db, ref[2])
