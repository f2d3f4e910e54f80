"""The MLP block's gradients: LayerNorm backward, and the activations' derivatives, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The forward definitions are ``oracle.layernorm`` and ``oracle.epilogue``; their
derivatives, written out:

* LayerNorm, per row, with xh = (x - mean) rs, g = dy gamma and means over the row
  (mean and rs depend on x):  dx = rs (g - mean(g) - xh mean(g xh)),
  dgamma = sum_rows dy xh, dbeta = sum_rows dy;
* GELU: gelu'(v) = Phi(v) + v phi(v), phi the standard normal density;
* SwiGLU h = silu(g) u over interleaved columns, s = sigmoid(g):
  dh/dg = u s (1 + g (1 - s)), dh/du = g s.
"""

from __future__ import annotations

import numpy as np
from scipy import special

from . import epilogue


def layernorm_backward(dy, x, gamma, mean, rs, dres=None):
    """(dx, dgamma, dbeta) at the given statistics."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    rs = np.asarray(rs, dtype=np.float64)[:, None]
    xh = (x - np.asarray(mean, dtype=np.float64)[:, None]) * rs
    g = dy * np.asarray(gamma, dtype=np.float64)[None, :]
    dx = rs * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def activation(pre, act):
    """[rows][cols] -> [rows][cols], SwiGLU [rows][cols / 2]."""
    return epilogue.epilogue_ref(pre, None, act)[1]


def activation_backward(dh, pre, act):
    """d pre [rows][cols] from dh [rows][cols], SwiGLU [rows][cols / 2]."""
    dh = np.asarray(dh, dtype=np.float64)
    if act == epilogue.ACT_NONE:
        return dh
    v = np.asarray(pre, dtype=np.float64)
    if act == epilogue.ACT_GELU:
        cdf = 0.5 * special.erfc(-v / np.sqrt(2.0))
        return dh * (cdf + v * np.exp(-0.5 * v * v) / np.sqrt(2.0 * np.pi))
    g, u = v[:, 0::2], v[:, 1::2]
    s, c = special.expit(g), special.expit(-g)
    d = np.empty_like(v)
    d[:, 0::2] = dh * u * s * (1.0 + g * c)
    d[:, 1::2] = dh * g * s
    return d
