"""GPU parity of fp8_gemm_residual against the oracle GEMM, oracle/epilogue.py and the residual in float64.

The bounds are those of the fused epilogue's tests (test_gpu_gemm_fused: the GEMM's own, one rounding of the bias add,
the activation's), plus one fp32 rounding of the residual add, and for a bf16 output one bf16 ulp."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from gpu_util import DEV, announce, gemm_bound, np_of  # noqa: E402
from oracle import epilogue as oe, gemm as og  # noqa: E402
from test_gpu_gemm_fused import _operands, _scal, _t, act_bound, check_values  # noqa: E402

NONE, GELU, SWIGLU = oe.ACT_NONE, oe.ACT_GELU, oe.ACT_SWIGLU
F32, BF16 = 0, 1
MODES = ["tensor", "block", "tile2", "mx"]


@pytest.fixture(scope="module")
def sq():
    import scaled_quantize_gemm_amd as m

    return m


def _residual(rng, M, N, out):
    r = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32))
    return r.to(torch.bfloat16 if out == BF16 else torch.float32)


def run_case(sq, mode, M, N, K, act, out, bias_kind, seed, rows=None, in_place=False):
    label = f"residual {mode} {(M, N, K)} act{act} out{out} bias={bias_kind}"
    announce(label)
    rng = np.random.default_rng(seed)
    dev, orc, bmode = _operands(sq, rng, mode, M, N, K)
    bias = None if bias_kind is None else _t(rng.standard_normal(N).astype(np.float32) * 0.5)
    if bias_kind == "bf16":
        bias = bias.to(torch.bfloat16)
    res = _residual(rng, M, N // 2 if act == SWIGLU else N, out)
    R = res.to(DEV)
    C = sq.fp8_gemm_residual(dev[0], 0, dev[1], dev[2], dev[3], 0, dev[4], dev[5], R, out, bias=bias, act=act,
                             C=R if in_place else None)
    torch.cuda.synchronize()
    assert (C.data_ptr() == R.data_ptr()) == in_place
    r = np.arange(M) if rows is None else rows
    Cr, S, G = og.gemm_ref(orc[0], 0, orc[1], orc[2], orc[3], 0, orc[4], orc[5], rows=r)
    pre, y = oe.epilogue_ref(Cr, None if bias is None else np_of(bias).astype(np.float64), act)
    e_pre = gemm_bound(S, G, K, bmode, False, Cr, Cr) + 2.0 ** -23 * (np.abs(pre) + 2.0 ** -10 * S)
    e_y = act_bound(pre, e_pre, act)
    want = y + np_of(res).astype(np.float64)[r]
    check_values(np_of(C)[r], want, e_y + 2.0 ** -24 * (np.abs(want) + e_y), out == BF16, label)
    return C


# every kernel's ragged edges, a single row, a single output pair, and the sizes around a token batch
SMALL = [(200, 264, 256), (65, 130, 384), (1, 2, 128), (3, 516, 128), (130, 64, 640)]
COMBOS = [(NONE, F32, "f32"), (GELU, BF16, "bf16"), (SWIGLU, BF16, "f32"), (NONE, BF16, None), (SWIGLU, F32, None)]


@pytest.mark.parametrize("combo", COMBOS, ids=str)
@pytest.mark.parametrize("mnk", SMALL, ids=str)
@pytest.mark.parametrize("mode", MODES)
def test_small(sq, mode, mnk, combo):
    act, out, bias = combo
    run_case(sq, mode, *mnk, act, out, bias, seed=sum(mnk) + 7 * act + 13 * out)


# a decoding step's tokens: 1 to 33 rows, N and K over narrow and wide weights, odd N
TOKENS = [(1, 768, 768), (1, 4096, 7168), (2, 770, 2304), (4, 517, 128), (7, 66, 4096), (8, 2304, 768), (15, 64, 1152),
          (16, 4096, 1024), (17, 300, 896), (31, 1028, 256), (32, 1500, 2048), (33, 260, 512), (16, 1, 256), (5, 3, 384)]


@pytest.mark.parametrize("mnk", TOKENS, ids=str)
@pytest.mark.parametrize("mode", MODES)
def test_tokens(sq, mode, mnk):
    act = NONE if mnk[1] % 2 else [NONE, GELU, SWIGLU][mnk[0] % 3]
    for out in (F32, BF16):
        run_case(sq, mode, *mnk, act, out, ["f32", "bf16", None][mnk[2] % 3], seed=sum(mnk), in_place=out == BF16)


# many tiles of the large kernels; N % 4 == 2 for the unaligned runs, and a blockwise split launch
LARGE = [("tensor", 4100, 4102, 256), ("mx", 2148, 4036, 384), ("block", 2085, 3002, 384), ("tile2", 1300, 4100, 256),
         ("tensor", 2048, 4096, 384), ("block", 2085, 4264, 256), ("tensor", 700, 2304, 256), ("tensor", 2048, 768, 512)]


@pytest.mark.parametrize("combo", COMBOS[:3], ids=str)
@pytest.mark.parametrize("case", LARGE, ids=str)
def test_large(sq, case, combo):
    mode, M, N, K = case
    act, out, bias = combo
    r = np.sort(np.random.default_rng(M + N).choice(M, 100, replace=False))
    r[-1] = M - 1
    run_case(sq, mode, M, N, K, act, out, bias, seed=M + 3 * act + out, rows=r, in_place=act == NONE)


@pytest.mark.parametrize("mode", MODES)
def test_zero_residual_equals_the_fused_gemm(sq, mode):
    """Beyond the token batches: with a residual of zeros, fp8_gemm_fused's values bit for bit (-0 aside)."""
    rng = np.random.default_rng(3)
    for M, N, K in ((264, 516, 512), (2052, 2304, 256)):
        dev, _, _ = _operands(sq, rng, mode, M, N, K)
        args = (dev[0], 0, dev[1], dev[2], dev[3], 0, dev[4], dev[5])
        bias = _t(rng.standard_normal(N).astype(np.float32))
        for act in (NONE, GELU, SWIGLU):
            zero = torch.zeros((M, N // 2 if act == SWIGLU else N), device=DEV)
            got = sq.fp8_gemm_residual(*args, zero, bias=bias, act=act)
            assert torch.equal(got, sq.fp8_gemm_fused(*args, out_dtype=sq.OUT_F32, bias=bias, act=act))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("M", [3, 200])
def test_k_zero(sq, mode, M):
    """K = 0: act(bias) + residual."""
    N = 260
    shape = {"tensor": ((1,), (1,)), "block": ((0, M), (3, 0)), "tile2": ((0, M), (0, N)), "mx": ((0, M), (0, N))}[mode]
    gran = {"tensor": (0, 0), "block": (1, 2), "tile2": (1, 1), "mx": (3, 3)}[mode]
    dt = torch.uint8 if mode == "mx" else torch.float32
    # an empty tensor has no address: one element's view keeps the pointers
    sa, sb = (torch.ones(max(1, int(np.prod(s))), dtype=dt, device=DEV)[:int(np.prod(s))].view(s) for s in shape)
    A, B = torch.empty((M, 0), dtype=torch.uint8, device=DEV), torch.empty((N, 0), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(4)
    bias, R = rng.standard_normal(N).astype(np.float32), rng.standard_normal((M, N)).astype(np.float32)
    if sa.data_ptr() == 0 or sb.data_ptr() == 0:
        with pytest.raises(sq.Fp8Error):
            sq.fp8_gemm_residual(A, 0, sa, gran[0], B, 0, sb, gran[1], _t(R), bias=_t(bias))
        return
    C = sq.fp8_gemm_residual(A, 0, sa, gran[0], B, 0, sb, gran[1], _t(R), bias=_t(bias))
    torch.cuda.synchronize()
    want = R + bias[None, :]
    assert np.array_equal(np_of(C), want)


def test_gradient_formats(sq):
    """E5M2 x E4M3 (a dgrad that joins the residual branch's gradient), exact inputs: every product and sum is a small
    whole number, so the result is exact on each route."""
    rng = np.random.default_rng(5)
    for M, N, K in ((5, 300, 256), (16, 4096, 512), (300, 520, 384), (2304, 2304, 256)):
        a, b = rng.integers(-4, 5, (M, K)), rng.integers(-4, 5, (N, K))
        A = torch.from_numpy(a.astype(np.float32)).to(torch.float8_e5m2).view(torch.uint8).to(DEV)
        B = torch.from_numpy(b.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
        R = rng.integers(-100, 101, (M, N))
        C = sq.fp8_gemm_residual(A, 1, _scal(1.0), 0, B, 0, _scal(0.5), 0, _t(R.astype(np.float32)))
        torch.cuda.synchronize()
        assert np.array_equal(np_of(C).astype(np.float64), 0.5 * (a @ b.T) + R), (M, N, K)


def test_accumulates_a_weight_gradient_in_place(sq):
    """Two micro-batches' wgrads into one fp32 buffer, exact inputs."""
    rng = np.random.default_rng(6)
    total, N, K = np.zeros((768, 512)), 512, 256
    acc = torch.zeros((768, 512), device=DEV)
    for _ in range(2):
        a, b = rng.integers(-4, 5, (768, K)), rng.integers(-4, 5, (N, K))
        A, B = (torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for v in (a, b))
        sq.fp8_gemm_residual(A, 0, _scal(1.0), 0, B, 0, _scal(1.0), 0, acc, C=acc)
        total += a @ b.T
    torch.cuda.synchronize()
    assert np.array_equal(np_of(acc).astype(np.float64), total)


def test_neighbours_stay_as_they_were(sq):
    """Rows behind the last token and memory behind C are not written."""
    rng = np.random.default_rng(7)
    for M, N in ((1, 517), (4, 768), (13, 260), (100, 514)):
        dev, _, _ = _operands(sq, rng, "tensor", M, N, 512)
        args = (dev[0], 0, dev[1], dev[2], dev[3], 0, dev[4], dev[5])
        R = _residual(rng, M, N, BF16).to(DEV)
        ref = sq.fp8_gemm_residual(*args, R)
        room = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
        sq.fp8_gemm_residual(*args, R, C=room[:M * N].view(M, N))
        torch.cuda.synchronize()
        assert torch.equal(room[:M * N].view(M, N), ref) and (room[M * N:] == 7).all()


def _random_cases(n=32, seed=31):
    rng = np.random.default_rng(seed)
    out = []
    for i in range(n):
        mode = MODES[i % 4]
        M = int(rng.integers(1, 40)) if i % 8 < 4 else int(rng.integers(40, 1101))
        N, act = int(rng.integers(1, 1101)), int(rng.integers(0, 3))
        N += N % 2 if act == SWIGLU else 0
        out.append((mode, M, N, 128 * int(rng.integers(1, 20)), act, int(rng.integers(0, 2)),
                    [None, "f32", "bf16"][int(rng.integers(0, 3))], 700 + i))
    return out


@pytest.mark.parametrize("case", _random_cases(), ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-a{c[4]}o{c[5]}")
def test_random_shapes(sq, case):
    mode, M, N, K, act, out, bias, seed = case
    run_case(sq, mode, M, N, K, act, out, bias, seed)
