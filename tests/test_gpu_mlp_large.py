"""The MLP block's operators where element offsets pass 32 bits (over 2^31 elements): the last rows and tiles equal those
of a small call on the same rows, and a reduction over all rows equals its parts."""

import pytest
import torch

pytestmark = pytest.mark.gpu

from gpu_util import DEV, announce  # noqa: E402

ROWS, COLS = 65664, 32768  # 2.15e9 elements; rows a multiple of 128
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sq():
    import scaled_quantize_gemm_amd as m

    return m


@pytest.fixture(scope="module")
def x():
    torch.cuda.empty_cache()
    g = torch.Generator(device=DEV).manual_seed(3)
    t = torch.empty((ROWS, COLS), dtype=BF, device=DEV)
    for i in range(0, ROWS, 8208):
        t[i:i + 8208] = torch.randn((8208, COLS), generator=g, device=DEV).to(BF)
    assert t.numel() > 1 << 31
    yield t
    torch.cuda.empty_cache()


def test_layernorm(sq, x):
    announce("layernorm past 2^31")
    g = torch.linspace(0.5, 1.5, COLS, device=DEV)
    mu, rs = torch.empty(2, ROWS, device=DEV).unbind(0)
    y = sq.fp8_layernorm(x, g, None, 1e-5, mu=mu, rsigma=rs)
    tail = slice(ROWS - 5, ROWS)
    assert torch.equal(y[tail], sq.fp8_layernorm(x[tail], g, None, 1e-5))
    dx, dg, db = sq.fp8_layernorm_backward(y, x, g, mu, rs)
    ref = sq.fp8_layernorm_backward(y[tail], x[tail], g, mu[tail], rs[tail])
    assert torch.equal(dx[tail], ref[0])
    want = torch.zeros(COLS, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for i in range(0, ROWS, 8208):
        part = y[i:i + 8208].double()
        want += part.sum(0)
        size += part.abs().sum(0)
    # at most rows / 4 + 64 additions one after another
    assert ((db.double() - want).abs() <= 2 * (ROWS / 4 + 64) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("tile", [False, True])
def test_activation(sq, x, tile):
    announce("activation past 2^31", tile)
    kw = dict(granularity=1) if tile else dict(scale=torch.full((1,), 100.0, device=DEV))
    q, qs, qT, qTs = sq.fp8_act_cast_transpose(x, sq.FP8_ACT_GELU, 0, **kw)
    for rows in (slice(ROWS - 128, ROWS), slice(0, 128)):
        r, rs, rT, rTs = sq.fp8_act_cast_transpose(x[rows], sq.FP8_ACT_GELU, 0, **kw)
        assert torch.equal(q[rows], r) and torch.equal(qT[:, rows], rT)
        if tile:
            assert torch.equal(qs[:, rows], rs) and torch.equal(qTs[rows.start // 128], rTs[0])


def test_gemm_residual(sq):
    announce("gemm residual past 2^31")
    torch.cuda.empty_cache()
    g = torch.Generator(device=DEV).manual_seed(4)
    M, N, K = ROWS, COLS, 128
    A, B = (torch.randint(-4, 5, (n, K), generator=g, device=DEV).float().to(torch.float8_e4m3fn).view(torch.uint8)
            for n in (M, N))
    one = torch.ones(1, device=DEV)
    R = torch.full((M, N), 3.0, dtype=BF, device=DEV)
    # whole numbers of at most 16 * 128 + 3: the fp32 sums are exact, bf16 rounds them once
    C = sq.fp8_gemm_residual(A, 0, one, 0, B, 0, one, 0, R, C=R)
    for rows in (slice(0, 64), slice(M - 64, M)):
        a, b = (t.view(torch.float8_e4m3fn).float() for t in (A[rows], B))
        assert torch.equal(C[rows], (a @ b.t() + 3).to(BF))
