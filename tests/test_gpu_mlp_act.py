"""GPU parity of fp8_act_cast_transpose and fp8_act_backward against float64 (oracle/epilogue.py, oracle/mlp.py).

The kernels evaluate in fp32, the oracle in float64, so a value v lies within e of the oracle's; the test then places
every amax, scale and code in the interval that e allows, as the LayerNorm + cast tests do.  e, with u = 2^-24
(act_math.h's operations counted; doubled at the end):
  Phi's tail: z one rounding, t = 1 / (1 + 0.3 z) 4 u, Q's nine steps on terms whose magnitudes add to 2.5 Q: 20 u, the
    fit 1 u, the exponential 2 u and its argument's 3 u times x^2/2, the products 3 u: (30 + 1.5 x^2) u of the tail, and
    below the smallest normal float the tail may be flushed; Phi = 1 - tail adds u;
  GELU one product; GELU' the density at (6 + 1.5 x^2) u of x phi(x) and one fma;
  sigmoid and 1 - sigmoid: argument 2 u |g|, exponential 2 u, reciprocal 3 u, product u: (6 + 2 |g|) u each;
  the products around them one rounding each."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from gpu_util import DEV, announce, np_of  # noqa: E402
from oracle import epilogue as oe, fp8 as ofp8, mlp as om, recipe as orc  # noqa: E402
from scipy import special  # noqa: E402
from test_gpu_layernorm import _codes_between, _f32_interval, _products  # noqa: E402

U, TINY = 2.0 ** -24, 2.0 ** -125
BF, F32 = torch.bfloat16, torch.float32
NONE, GELU, SWIGLU = oe.ACT_NONE, oe.ACT_GELU, oe.ACT_SWIGLU


@pytest.fixture(scope="module")
def sq():
    import scaled_quantize_gemm_amd as m

    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def _rand(rng, shape, std=1.0, dtype=F32):
    return torch.from_numpy((std * rng.standard_normal(shape)).astype(np.float32)).to(dtype)


def _e_cdf(v):
    tail = 0.5 * special.erfc(np.abs(v) / np.sqrt(2.0))
    return (30 + 1.5 * v * v) * U * tail + TINY + U


def _e_cdf_signed(v):
    """Without the 1 - tail rounding where v < 0."""
    return _e_cdf(v) - np.where(v < 0, U, 0.0)


def forward_bound(pre, act):
    h = om.activation(pre, act)
    if act == GELU:
        return h, 2 * (np.abs(pre) * _e_cdf_signed(pre) + U * np.abs(h)) + TINY
    g = pre[:, 0::2]
    return h, 2 * (10 + 2 * np.abs(g)) * U * np.abs(h) + TINY * (1 + np.abs(pre[:, 1::2]))


def backward_bound(dh, pre, act):
    d = om.activation_backward(dh, pre, act)
    if act == NONE:
        return d, np.zeros_like(d)
    a = np.abs(dh)
    if act == GELU:
        dens = np.abs(pre) * np.exp(-0.5 * pre * pre) / np.sqrt(2 * np.pi)
        return d, 2 * (a * (_e_cdf_signed(pre) + (7 + 1.5 * pre * pre) * U * dens + 2 * U) + U * np.abs(d)) + TINY
    g, u = pre[:, 0::2], pre[:, 1::2]
    s, c = special.expit(g), special.expit(-g)
    k = (6 + 2 * np.abs(g)) * U
    e = np.empty_like(d)
    inner = np.abs(1 + g * c)
    e[:, 0::2] = a * np.abs(u) * s * ((k + 3 * U) * inner + (k + U) * np.abs(g) * c + U * inner)
    e[:, 1::2] = a * np.abs(g) * s * (k + 3 * U)
    return d, 2 * e + TINY * (1 + np.abs(d))


def check_cast(out, h, e, fmt, tile, scale, slot, label, slot0=0.0):
    """q, q_scale_inv, qT, qT_scale_inv of a result known as h within e."""
    q, qs, qT, qTs = (None if t is None else np_of(t) for t in out)
    assert q.shape == h.shape and qT.shape == h.T.shape
    if not tile:
        assert qs is None and qTs is None
        assert np.array_equal(qT, q.T), f"{label}: qT is not q transposed"
        s = np.float64(np.float32(scale))
        _codes_between(q, (h - e) * s, (h + e) * s, fmt, label)
        if slot is not None:
            lo = max(slot0, float((np.abs(h) - e).max(initial=0.0)))
            hi = max(slot0, float((np.abs(h) + e).max(initial=0.0)))
            assert lo * (1 - U) <= float(slot) <= hi * (1 + U), (label, float(slot), lo, hi)
        return
    for codes, sinv, v, ev, name in ((q, qs, h, e, "q"), (qT, qTs, h.T, e.T, "qT")):
        n, m = v.shape
        alo, ahi = _f32_interval(np.maximum(np.abs(v) - ev, 0).reshape(n, m // 128, 128).max(axis=2),
                                 (np.abs(v) + ev).reshape(n, m // 128, 128).max(axis=2))
        assert (alo > 0).all(), "zero runs are checked elsewhere"
        s_hi, si_lo = orc.current_scale(alo, fmt)
        s_lo, si_hi = orc.current_scale(ahi, fmt)
        got = sinv.T
        assert ((si_lo <= got) & (got <= si_hi)).all(), (label, name, "scale_inv")
        slo, shi = (np.repeat(np.asarray(s, np.float64), 128, axis=1) for s in (s_lo, s_hi))
        _codes_between(codes, *_products(v - ev, v + ev, slo, shi), fmt, f"{label} {name}")


def check_dbias(dbias, d, e, rows, label):
    n = min(rows, rows / 4 + 160)
    bound = 2 * n * U * (np.abs(d) + e).sum(axis=0) + e.sum(axis=0)
    err = np.abs(f64(dbias) - d.sum(axis=0))
    assert (err <= bound).all(), (label, "dbias", (err - bound).max())


def run(sq, backward, R, C, act, fmt, tile, dtype, seed, std=1.0, amax0=0.0, pre=None, dh=None, want_dbias=True):
    label = f"{'bwd' if backward else 'fwd'} {R}x{C} act{act} fmt{fmt} {'tile' if tile else 'tensor'} {dtype}"
    announce(label)
    rng = np.random.default_rng(seed)
    if pre is None and act != NONE:
        pre = _rand(rng, (R, C), std, dtype)
    width = C // 2 if act == SWIGLU else C
    if backward and dh is None:
        dh = _rand(rng, (R, width), 1e-3, dtype)
    # a scale under which the largest results saturate
    scale = ofp8.FMAX[fmt] / (3e-3 if backward else 3.0)
    slot = None if tile else torch.full((1,), amax0, device=DEV)
    kw = dict(granularity=sq.FP8_SCALE_TILE_1x128) if tile else dict(
        granularity=sq.FP8_SCALE_TENSOR, scale=torch.tensor([scale], dtype=F32, device=DEV), amax_slot=slot)
    p = None if pre is None else pre.to(DEV)
    if backward:
        out = sq.fp8_act_backward(dh.to(DEV), p, act, fmt, want_dbias=want_dbias, **kw)
        torch.cuda.synchronize()
        v, e = backward_bound(f64(dh), None if pre is None else f64(pre), act)
        if want_dbias:
            check_dbias(out[4], v, e, R, label)
        else:
            assert out[4] is None
    else:
        out = sq.fp8_act_cast_transpose(p, act, fmt, **kw)
        torch.cuda.synchronize()
        v, e = forward_bound(f64(pre), act)
    check_cast(out[:4], v, e, fmt, tile, scale, None if slot is None else np_of(slot)[0], label, amax0)
    return out


# per tensor: one element, one row, one column, widths and heights around 4, 8, 64 and 128, odd ones
RAGGED = [(1, 2), (1, 768), (300, 2), (5, 6), (7, 130), (64, 64), (66, 72), (128, 256), (130, 264), (127, 254),
          (129, 1026), (260, 136), (1000, 514)]


@pytest.mark.parametrize("shape", RAGGED, ids=str)
@pytest.mark.parametrize("act", [GELU, SWIGLU])
def test_forward_tensor(sq, shape, act):
    for fmt, dtype in ((0, BF), (1, F32)):
        run(sq, False, *shape, act, fmt, False, dtype, sum(shape) + fmt, std=1.5)


@pytest.mark.parametrize("shape", RAGGED, ids=str)
@pytest.mark.parametrize("act", [NONE, GELU, SWIGLU])
def test_backward_tensor(sq, shape, act):
    for fmt, dtype in ((1, BF), (0, F32)):
        run(sq, True, *shape, act, fmt, False, dtype, sum(shape) + fmt, std=1.5)


@pytest.mark.parametrize("cols", [1, 3, 131, 255])
def test_odd_columns(sq, cols):
    run(sq, False, 37, cols, GELU, 0, False, BF, cols)
    run(sq, True, 37, cols, GELU, 1, False, F32, cols)
    run(sq, True, 38, cols, NONE, 1, False, BF, cols)


@pytest.mark.parametrize("shape", [(128, 256), (256, 512), (384, 1280)], ids=str)
@pytest.mark.parametrize("act", [NONE, GELU, SWIGLU])
@pytest.mark.parametrize("fmt,dtype", [(0, BF), (1, BF), (0, F32), (1, F32)])
def test_tile(sq, shape, act, fmt, dtype):
    if act != NONE:
        run(sq, False, *shape, act, fmt, True, dtype, sum(shape) + act, std=1.5)
    run(sq, True, *shape, act, fmt, True, dtype, sum(shape) + act, std=1.5)


# many tiles: grids that are capped, and blocks that take several tiles
@pytest.mark.parametrize("act", [NONE, GELU, SWIGLU])
def test_many_tiles(sq, act):
    if act != NONE:
        run(sq, False, 2048, 3584, act, 0, False, BF, act)
        run(sq, False, 1280, 2304, act, 0, True, BF, act)
    run(sq, True, 2048, 3584, act, 1, False, BF, act)
    run(sq, True, 1280, 2304, act, 0, True, BF, act)
    run(sq, True, 1533, 2310, act, 1, False, BF, act)


def test_wide_values(sq):
    """Pre-activations across the whole range that matters: the tails of Phi and of the sigmoid, and far beyond."""
    v = torch.cat([torch.linspace(-14, 14, 128 * 127), torch.tensor([0.0, -0.0, 100.0, -100.0, 3e4, -3e4, 1e-30, -1e-30]).repeat(16)])
    pre = v.view(128, 128)
    for act in (GELU, SWIGLU):
        run(sq, False, 128, 128, act, 0, False, F32, 3, pre=pre)
        run(sq, True, 128, 128, act, 1, False, F32, 4, pre=pre)


def test_amax_accumulates_and_dbias_may_be_left_out(sq):
    run(sq, False, 130, 264, GELU, 0, False, BF, 5, amax0=1e6)
    run(sq, True, 130, 264, SWIGLU, 1, False, BF, 6, amax0=1e6, want_dbias=False)
    rng = np.random.default_rng(7)
    pre, one = _rand(rng, (130, 264), dtype=BF).to(DEV), torch.ones(1, device=DEV)
    q, _, qT, _ = sq.fp8_act_cast_transpose(pre, GELU, 0, scale=one)  # no slot
    assert torch.equal(qT, q.t())


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_non_finite_elements(sq, backward, tile):
    """A NaN gives the NaN code (and, in runs, scale 1 for its runs) and stays in its own element; in the amax it
    propagates."""
    rng = np.random.default_rng(8)
    pre = _rand(rng, (128, 128))
    at = (5, 17)
    bad = pre.clone()
    bad[at] = float("nan")
    kw = dict(granularity=1) if tile else dict(scale=torch.full((1,), 100.0, device=DEV))
    slot = torch.zeros(1, device=DEV)
    if not tile:
        kw["amax_slot"] = slot
    dh = _rand(rng, (128, 128)).to(DEV)

    def f(p):
        if backward:
            return sq.fp8_act_backward(dh, p.to(DEV), GELU, 1, **kw)
        return sq.fp8_act_cast_transpose(p.to(DEV), GELU, 1, **kw)

    ref, got = f(pre), f(bad)
    torch.cuda.synchronize()
    q, qT = np_of(got[0]), np_of(got[2])
    assert q[at] & 0x7F == 0x7F and qT[at[::-1]] & 0x7F == 0x7F
    same = np.ones((128, 128), bool)
    if tile:
        same[at[0], :] = False
        assert np_of(got[1])[0, at[0]] == 1.0 and np_of(got[3])[0, at[1]] == 1.0
    else:
        same[at] = False
        assert np.isnan(np_of(slot)[0])
    assert np.array_equal(q[same], np_of(ref[0])[same])
    same = np.ones((128, 128), bool)
    if tile:
        same[at[1], :] = False
    else:
        same[at[::-1]] = False
    assert np.array_equal(qT[same], np_of(ref[2])[same])
    if backward:
        b = np_of(got[4])
        assert np.isnan(b[at[1]]) and np.array_equal(np.delete(b, at[1]), np.delete(np_of(ref[4]), at[1]))


@pytest.mark.parametrize("fmt", [0, 1])
def test_no_activation_equals_the_cast_transposes(sq, fmt):
    """FP8_ACT_NONE casts dh itself: the codes, scales and amax of fp8_cast_transpose and of its blockwise form."""
    rng = np.random.default_rng(9)
    for R, C in ((256, 384), (100, 200), (33, 517)):
        dh, s = _rand(rng, (R, C), 1e-3, BF).to(DEV), torch.full((1,), 1e5, device=DEV)
        a, b = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        got = sq.fp8_act_backward(dh, None, NONE, fmt, scale=s, amax_slot=a)
        q, qT = sq.fp8_cast_transpose(dh, fmt, s, amax_slot=b)
        assert torch.equal(got[0], q) and torch.equal(got[2], qT) and torch.equal(a, b)
        if R % 128 == 0:
            got = sq.fp8_act_backward(dh, None, NONE, fmt, granularity=1)
            for x, y in zip(got[:4], sq.fp8_cast_transpose_blockwise(dh, fmt, 1)):
                assert torch.equal(x, y)


def test_zero_runs(sq):
    """Runs of zeros take scale 1; a zero gradient gives zero codes and a zero bias gradient."""
    pre = torch.zeros((128, 256), dtype=BF, device=DEV)
    q, qs, qT, qTs = sq.fp8_act_cast_transpose(pre, GELU, 0, granularity=1)
    assert not (q & 0x7F).any() and not (qT & 0x7F).any() and (qs == 1).all() and (qTs == 1).all()
    out = sq.fp8_act_backward(torch.zeros((128, 128), dtype=BF, device=DEV), pre + 1, SWIGLU, 1, granularity=1)
    assert not (out[0] & 0x7F).any() and (out[1] == 1).all() and (out[3] == 1).all() and not out[4].any()


def test_infinite_pre_activations(sq):
    """GELU's limits at the infinities: +inf saturates and is the amax, -inf gives zero; nothing turns into NaN."""
    pre = torch.ones((128, 256))
    pre[3, 7], pre[4, 8] = float("inf"), -float("inf")
    for dtype in (BF, F32):
        slot = torch.zeros(1, device=DEV)
        q, _, qT, _ = sq.fp8_act_cast_transpose(pre.to(dtype).to(DEV), GELU, 0, scale=torch.ones(1, device=DEV), amax_slot=slot)
        assert q[3, 7] == 0x7E and q[4, 8] & 0x7F == 0 and torch.equal(qT, q.t()) and torch.isinf(slot).all()
        q, qs, qT, qTs = sq.fp8_act_cast_transpose(pre.to(dtype).to(DEV), GELU, 0, granularity=1)
        assert q[3, 7] == 0x7E and qT[7, 3] == 0x7E and qs[0, 3] == 1 and qTs[0, 7] == 1 and qs[0, 4] != 1
        # a finite value under scale 1 beside the infinity: gelu(1) = 0.841 -> 0.8125 = 0x35
        assert q[3, 8] == 0x35 and qT[7, 4] == 0x35


def test_empty(sq):
    one = torch.ones(1, device=DEV)
    none = torch.empty((0, 256), dtype=BF, device=DEV)
    q, _, qT, _ = sq.fp8_act_cast_transpose(none, SWIGLU, 0, scale=one)
    assert q.shape == (0, 128) and qT.shape == (128, 0)
    dbias = torch.full((256,), 3.0, device=DEV)
    sq.fp8_act_backward(none[:, :128].contiguous(), none, SWIGLU, 0, scale=one, dbias=dbias)
    assert not dbias.any()
    out = sq.fp8_act_backward(torch.empty((5, 0), device=DEV), None, NONE, 0, scale=one)
    assert out[0].shape == (5, 0) and out[4].numel() == 0


def test_neighbours_stay_as_they_were(sq):
    rng = np.random.default_rng(10)
    for R, C in ((130, 264), (127, 250)):
        pre, dh, one = _rand(rng, (R, C), dtype=BF).to(DEV), _rand(rng, (R, C // 2), dtype=BF).to(DEV), torch.ones(1, device=DEV)
        ref = sq.fp8_act_backward(dh, pre, SWIGLU, 1, scale=one)
        torch.cuda.synchronize()
        q, qT = (torch.full((R * C + 64,), 0xAB, dtype=torch.uint8, device=DEV) for _ in range(2))
        db = torch.full((C + 5,), 9.0, device=DEV)
        ws = torch.full((sq.fp8_act_backward_workspace(R, C) + 64,), 0xFF, dtype=torch.uint8, device=DEV)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            sq.fp8_act_backward(dh, pre, SWIGLU, 1, scale=one, q=q[:R * C].view(R, C), qT=qT[:R * C].view(C, R),
                                dbias=db[:C], workspace=ws[:-64])
        st.synchronize()
        assert torch.equal(q[:R * C].view(R, C), ref[0]) and torch.equal(qT[:R * C].view(C, R), ref[2])
        assert torch.equal(db[:C], ref[4]) and (db[C:] == 9).all() and (ws[-64:] == 0xFF).all()
        assert (q[R * C:] == 0xAB).all() and (qT[R * C:] == 0xAB).all()
