"""Oracle for the channels-last group norm with an activation or a gate — TEST INFRASTRUCTURE ONLY
(the same import rules as the rest of ``oracle/``).  Plain fp64 numpy from the definition: for a
sample and a group of channels, over its M values,

    xhat = (x - mean) / sqrt(var + eps),  u = xhat w + b,  y = act(u)  or  u act(gate)

and with dhat the gradient of xhat, dx = rstd (dhat - E[dhat] - xhat E[dhat xhat])."""
from __future__ import annotations

import numpy as np

from .selective import sigmoid


def _act(v, silu):
    return v * sigmoid(v) if silu else v


def _slope(v, silu):
    if not silu:
        return np.ones_like(v)
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def _parts(x, groups, weight, bias, eps):
    x = np.asarray(x, np.float64)
    C = x.shape[-1]
    grouped = x.reshape(x.shape[0], -1, groups, C // groups)
    mean = grouped.mean((1, 3))
    rstd = 1.0 / np.sqrt(((grouped - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    hat = ((grouped - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    w = np.ones(C) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    return x, mean, rstd, hat, w, hat * w + b


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, silu=False, gate=None):
    """(y, mean, rstd)."""
    _, mean, rstd, _, _, u = _parts(x, groups, weight, bias, eps)
    y = _act(u, silu) if gate is None else u * _act(np.asarray(gate, np.float64), silu)
    return y, mean, rstd


def group_norm_backward(dy, x, groups, weight=None, bias=None, eps=1e-5, silu=False, gate=None):
    """(dx, dweight, dbias, dgate or None)."""
    x, _, rstd, hat, w, u = _parts(x, groups, weight, bias, eps)
    dy = np.asarray(dy, np.float64)
    dgate = None
    if gate is None:
        du = dy * _slope(u, silu)
    else:
        gate = np.asarray(gate, np.float64)
        du, dgate = dy * _act(gate, silu), dy * u * _slope(gate, silu)
    over = tuple(range(x.ndim - 1))
    shape = (x.shape[0], -1, groups, x.shape[-1] // groups)
    dhat, h = (du * w).reshape(shape), hat.reshape(shape)
    dx = rstd[:, None, :, None] * (dhat - dhat.mean((1, 3), keepdims=True) -
                                   h * (dhat * h).mean((1, 3), keepdims=True))
    return dx.reshape(x.shape), (du * hat).sum(over), du.sum(over), dgate
