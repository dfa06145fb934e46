"""Oracle for the norms before and after a block with its gate and residual scale — TEST
INFRASTRUCTURE ONLY (the same import rules as the rest of ``oracle/``).  Plain fp64 numpy from the
definition, rows over the last axis:

    n = h / sqrt(E[h^2] + eps) post,  z = n act(gate),  x' = x + alpha z,  y = x' / sqrt(E[x'^2] + eps) w

and for u = v / sqrt(E[v^2] + eps) with gradient du: dv = rstd (du - u E[du u])."""
from __future__ import annotations

import numpy as np

from .selective import sigmoid


def _norm(v, eps):
    rstd = 1.0 / np.sqrt((v ** 2).mean(-1, keepdims=True) + eps)
    return v * rstd, rstd


def _back(du, u, rstd):
    return rstd * (du - u * (du * u).mean(-1, keepdims=True))


def _parts(x, h, weight, post_norm, post, gate, silu, scale, residual_scale, eps):
    f = lambda t, one=1.0: one if t is None else np.asarray(t, np.float64)  # noqa: E731
    x = f(x)
    h = np.zeros_like(x) if h is None else f(h)
    hat, rstd1 = _norm(h, eps) if post_norm else (h, np.ones(h.shape[:-1] + (1,)))
    gate, post, w = f(gate), f(post), f(weight)
    act = gate * sigmoid(gate) if silu and np.ndim(gate) else gate
    alpha = residual_scale * f(scale)
    z = hat * post * act
    out = x + alpha * z
    hat2, rstd2 = _norm(out, eps)
    return out, hat2 * w, rstd1, rstd2, hat, hat2, post, w, gate, act, alpha, z


def block_norm(x, h=None, weight=None, post_norm=False, post=None, gate=None, silu=False,
               scale=None, residual_scale=1.0, eps=1e-5):
    """(x', y, post_rstd, rstd)."""
    out, y, rstd1, rstd2 = _parts(x, h, weight, post_norm, post, gate, silu, scale,
                                  residual_scale, eps)[:4]
    return out, y, rstd1[..., 0], rstd2[..., 0]


def block_norm_backward(dy, dx, x, h=None, weight=None, post_norm=False, post=None, gate=None,
                        silu=False, scale=None, residual_scale=1.0, eps=1e-5):
    """Gradients as a dict: dx, dh, dgate, dweight, dpost, dscale."""
    _, _, rstd1, rstd2, hat, hat2, post, w, gate, act, alpha, z = _parts(
        x, h, weight, post_norm, post, gate, silu, scale, residual_scale, eps)
    f = lambda t: 0.0 if t is None else np.asarray(t, np.float64)  # noqa: E731
    dR = f(dx) + (0.0 if dy is None else _back(f(dy) * w, hat2, rstd2))
    over = tuple(range(hat.ndim - 1))
    dz = alpha * dR
    dn = dz * act
    slope = 1.0
    if silu and np.ndim(gate):
        s = sigmoid(gate)
        slope = s * (1.0 + gate * (1.0 - s))
    dh = _back(dn * post, hat, rstd1) if post_norm else dn * post
    return dict(dx=dR, dh=dh, dgate=dz * hat * post * slope, dweight=(f(dy) * hat2).sum(over),
                dpost=(dn * hat).sum(over), dscale=(dR * z).sum(over) * residual_scale)
