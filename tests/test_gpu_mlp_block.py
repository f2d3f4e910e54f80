"""A training step of the MLP block with every operator in its place (norm -> FC1 + SwiGLU -> FC2 + residual, and back),
against float64 and against differences; captured as a graph, its replays equal the eager step bit for bit; two steps on
two streams at once equal the same steps one after another."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from gpu_util import DEV, announce  # noqa: E402
from oracle import epilogue as oe, layernorm as oln, mlp as om  # noqa: E402

EPS = 1e-5
E4, E5 = 0, 1


@pytest.fixture(scope="module")
def sq():
    import scaled_quantize_gemm_amd as m

    return m


class MlpBlock:
    """x + FC2(swiglu(FC1(layernorm(x)))), hybrid delayed scaling.  Slots: xn, w1, h, w2 (E4M3), dy, dpre (E5M2)."""

    def __init__(self, sq, tokens, width, inner, seed=0):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        rnd = lambda *s, std=1.0: (std * torch.randn(*s, generator=g))  # noqa: E731
        self.sq = sq
        self.x, self.dy = rnd(tokens, width).to(bf).to(DEV), rnd(tokens, width, std=0.01).to(bf).to(DEV)
        self.w1 = rnd(2 * inner, width, std=width ** -0.5).to(bf).to(DEV)
        self.w2 = rnd(width, inner, std=inner ** -0.5).to(bf).to(DEV)
        self.gamma, self.beta = (1 + rnd(width, std=0.1)).to(DEV), rnd(width, std=0.1).to(DEV)
        self.b1, self.b2 = rnd(2 * inner, std=0.1).to(DEV), rnd(width, std=0.1).to(DEV)
        self.state = sq.DelayedScalingState([E4, E4, E4, E4, E5, E5], history_len=4, device=DEV)
        self.mu, self.rs = torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV)
        self.aux = torch.empty((tokens, 2 * inner), dtype=bf, device=DEV)

    def forward(self, x=None):
        sq, T = self.sq, self.sq.FP8_SCALE_TENSOR
        x = self.x if x is None else x
        slots = [self.state.slot(i) for i in range(6)]
        (sx, ax, ix), (s1, a1, i1), (sh, ah, ih), (s2, a2, i2) = slots[:4]
        xn = sq.fp8_layernorm(x, self.gamma, self.beta, EPS, mu=self.mu, rsigma=self.rs)
        self.qx, self.qxT = sq.fp8_cast_transpose(xn, E4, sx, ax)
        self.q1, self.q1T = sq.fp8_cast_transpose(self.w1, E4, s1, a1)
        self.q2, self.q2T = sq.fp8_cast_transpose(self.w2, E4, s2, a2)
        self.pre = sq.fp8_gemm_fused(self.qx, E4, ix, T, self.q1, E4, i1, T, sq.OUT_BF16, bias=self.b1)
        self.qh, _, self.qhT, _ = sq.fp8_act_cast_transpose(self.pre, sq.FP8_ACT_SWIGLU, E4, scale=sh, amax_slot=ah)
        return sq.fp8_gemm_residual(self.qh, E4, ih, T, self.q2, E4, i2, T, x, bias=self.b2)

    def backward(self):
        sq, T = self.sq, self.sq.FP8_SCALE_TENSOR
        ix, i1, ih, i2 = (self.state.slot(i)[2] for i in range(4))
        sy, ay, iy = self.state.slot(4)
        sp, ap, ip = self.state.slot(5)
        qy, _, qyT, _, db2 = sq.fp8_act_backward(self.dy, None, sq.FP8_ACT_NONE, E5, scale=sy, amax_slot=ay)
        dh = sq.fp8_gemm(qy, E5, iy, T, self.q2T, E4, i2, T, sq.OUT_BF16)
        dw2 = sq.fp8_gemm(qyT, E5, iy, T, self.qhT, E4, ih, T, sq.OUT_F32)
        qp, _, qpT, _, db1 = sq.fp8_act_backward(dh, self.pre, sq.FP8_ACT_SWIGLU, E5, scale=sp, amax_slot=ap)
        dxn = sq.fp8_gemm(qp, E5, ip, T, self.q1T, E4, i1, T, sq.OUT_BF16)
        dw1 = sq.fp8_gemm(qpT, E5, ip, T, self.qxT, E4, ix, T, sq.OUT_F32)
        dx, dgamma, dbeta = sq.fp8_layernorm_backward(dxn, self.x, self.gamma, self.mu, self.rs, dres=self.dy)
        return dict(dx=dx, dgamma=dgamma, dbeta=dbeta, dw1=dw1, db1=db1, dw2=dw2, db2=db2)

    def step(self):
        y = self.forward()
        grads = self.backward()
        self.state.update()
        return {"y": y, **grads, "history": self.state.amax_history, "scale": self.state.scale}


def f64(t):
    return t.detach().cpu().double().numpy()


def _reference(b):
    """The block in float64 without any cast, forward and backward."""
    x, g, be, dy = f64(b.x), f64(b.gamma), f64(b.beta), f64(b.dy)
    w1, w2, b1, b2 = f64(b.w1), f64(b.w2), f64(b.b1), f64(b.b2)
    xn, mean, rs = oln.layernorm_ref(x, g, be, EPS)
    pre = xn @ w1.T + b1
    h = om.activation(pre, oe.ACT_SWIGLU)
    dh = dy @ w2
    dpre = om.activation_backward(dh, pre, oe.ACT_SWIGLU)
    dx, dgamma, dbeta = om.layernorm_backward(dpre @ w1, x, g, mean, rs, dy)
    return dict(y=x + h @ w2.T + b2, dx=dx, dgamma=dgamma, dbeta=dbeta, dw1=dpre.T @ xn, db1=dpre.sum(0), dw2=dy.T @ h,
                db2=dy.sum(0))


# In the 2-norm.  An E4M3 cast is off by 2^-4 of a value at most, evenly spread 2^-4 / sqrt 3 = 0.036 at the top of a
# binade and half that at its bottom, 0.027 over the binade's values; E5M2 twice that; what underflows adds little
# under scales that fill the range.  Independent errors add in squares.  E4M3 = 0.027, E5M2 = 0.054:
#   pre: two casts, 0.038.  h: pre's error through silu(g) u, at most 1.1 sqrt 2 of it in the mean, and a cast: 0.065.
#   y (without the stream x, which is exact): h and w2: 0.070.     dw2: dy and h: sqrt(0.054^2 + 0.065^2) = 0.085.
#   dh: 0.060.  dpre: dh's, pre's through the second derivative (0.06), its own cast: 0.10.
#   dxn, and dx beside the exact residual: dpre and w1: 0.105.  dw1: dpre and xn: 0.105.  db1: dpre before its cast, as
#   independent errors over the rows: 0.085.  dgamma, dbeta: sums over the rows of dxn: 0.105.  db2: exact but for fp32.
BOUND = dict(y=0.070, dx=0.105, dgamma=0.105, dbeta=0.105, dw1=0.105, db1=0.085, dw2=0.085, db2=1e-5)


@pytest.mark.parametrize("tokens,width,inner", [(256, 256, 384), (384, 512, 640)])
def test_step_against_float64(sq, tokens, width, inner):
    announce("mlp block", tokens, width, inner)
    b = MlpBlock(sq, tokens, width, inner)
    for _ in range(2):  # the second step runs under the first one's scales
        out = b.step()
    torch.cuda.synchronize()
    ref = _reference(b)
    x, dy = f64(b.x), f64(b.dy)
    past = dict(y=x, dx=dy)  # what passes the block unchanged: the error is that of the rest
    for k, tol in BOUND.items():
        off = np.linalg.norm(f64(out[k]) - ref[k]) / np.linalg.norm(ref[k] - past.get(k, 0.0))
        # y and dx are rounded to bf16 as a whole, by at most 2^-8 of them
        room = 2.0 ** -8 * np.linalg.norm(ref[k]) / np.linalg.norm(ref[k] - past[k]) if k in past else 0.0
        print(f"[mlp] {k} {off:.4f} of {tol + room:.4f}", flush=True)
        assert off <= tol + room, (k, off)


def test_gradient_against_differences(sq):
    """dx . v against (L(x + t v) - L(x - t v)) / 2t with L = <y, dy> in float64 over the block's own fp8 forward.  The
    casts make y a staircase: over a step t = 1/4 of the input's spread many stairs are passed, each value's error is
    independent, and the two sides agree like dx itself does, beside the curvature of the block over that step."""
    b = MlpBlock(sq, 256, 256, 384, seed=3)
    for _ in range(2):
        out = b.step()
    dx = f64(out["dx"])
    want, got, t = [], [], 0.0625
    for k in range(6):
        # along the gradient itself with random signs kept for a third of the rows: a direction with a clear derivative
        rng = np.random.default_rng(k)
        rows = rng.random((256, 1)) < 0.33
        v = np.where(rows, dx / np.sqrt((dx ** 2).mean()), 0.0)
        xp, xm = ((b.x.double() + s * t * torch.from_numpy(v).to(DEV)).to(torch.bfloat16) for s in (1, -1))
        real = f64(xp) - f64(xm)  # the step that bf16 left of it
        L = [float((f64(b.forward(x)) * f64(b.dy)).sum()) for x in (xp, xm)]
        got.append(L[0] - L[1])
        want.append(float((dx * real).sum()))
    got, want = np.array(got), np.array(want)
    print("[mlp] differences", got / want, flush=True)
    # 0.105 (dx above) + the forward casts' share of a difference of two y: 0.070 sqrt 2 of the difference's own norm,
    # spread over 256 x 256 independent values, and a curvature of t^2 / 6 times order 1: 0.11 + 0.01 + 0.01
    assert np.abs(got / want - 1).max() < 0.13


def test_graph_replays_match_eager(sq):
    b = MlpBlock(sq, 512, 768, 896, seed=1)
    st = b.state
    start = [t.clone() for t in (st.amax_history, st.scale, st.scale_inv)]
    eager = []
    for _ in range(3):
        out = b.step()
        torch.cuda.synchronize()
        eager.append({k: v.clone() for k, v in out.items()})
    for dst, src in zip((st.amax_history, st.scale, st.scale_inv), start):
        dst.copy_(src)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.step()
    torch.cuda.synchronize()
    for dst, src in zip((st.amax_history, st.scale, st.scale_inv), start):
        dst.copy_(src)
    for k in range(3):
        announce("mlp graph replay", k)
        g.replay()
        torch.cuda.synchronize()
        for name, v in out.items():
            assert torch.equal(v.view(torch.uint8), eager[k][name].view(torch.uint8)), (k, name)
        torch.ones(1 << 20, device=DEV).mul_(2.0).sum().item()


def test_two_graphs_of_two_blocks_interleaved(sq):
    """Two captured steps replayed in turn, workspaces and all from each graph's own pool."""
    blocks = [MlpBlock(sq, 256, 256, 384, seed=s) for s in (1, 2)]
    want, graphs, outs = [], [], []
    for b in blocks:
        st = b.state
        start = [t.clone() for t in (st.amax_history, st.scale, st.scale_inv)]
        b.step()
        want.append([{k: v.clone() for k, v in b.step().items()}, {k: v.clone() for k, v in b.step().items()}])
        for dst, src in zip((st.amax_history, st.scale, st.scale_inv), start):
            dst.copy_(src)
        b.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        keep = [t.clone() for t in (st.amax_history, st.scale, st.scale_inv)]
        with torch.cuda.graph(g):
            outs.append(b.step())
        for dst, src in zip((st.amax_history, st.scale, st.scale_inv), keep):
            dst.copy_(src)
        graphs.append(g)
    for k in range(2):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            for name, v in out.items():
                assert torch.equal(v.view(torch.uint8), w[k][name].view(torch.uint8)), (k, name)


def test_two_streams_at_once(sq):
    blocks = [MlpBlock(sq, 384, 512, 640, seed=s) for s in (4, 5)]
    twins = [MlpBlock(sq, 384, 512, 640, seed=s) for s in (4, 5)]
    want = []
    for b in twins:
        b.step()
        want.append({k: v.clone() for k, v in b.step().items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [None, None]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        for i, (b, s) in enumerate(zip(blocks, streams)):
            with torch.cuda.stream(s):
                got[i] = b.step()
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        for name, v in o.items():
            assert torch.equal(v.view(torch.uint8), w[name].view(torch.uint8)), name
