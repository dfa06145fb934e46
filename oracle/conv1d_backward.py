"""Oracle for the gradient of the causal convolution (``oracle.conv1d``) — TEST INFRASTRUCTURE ONLY.
Plain fp64 numpy: with x~ the W - 1 inputs before a sequence and then its inputs, u[t] = bias +
sum_i w[i] x~[t + i], y = act(u), and the last W - 1 entries of x~ as the final state,

    du = dy act'(u),  dx~[e] = sum_i w[i] du[e - i] (+ dfinal),  dw[i] = sum_t du[t] x~[t + i]."""
from __future__ import annotations

import numpy as np

from .selective import sigmoid


def causal_conv1d_backward(x, weight, dy, bias=None, initial=None, dfinal=None, cu=None,
                           silu=False):
    """(dx, dweight, dbias, dinitial); initial, dfinal, dinitial [N, W - 1, C]."""
    f = lambda t: None if t is None else np.asarray(t, np.float64)  # noqa: E731
    x, w, dy, bias, initial, dfinal = map(f, (x, weight, dy, bias, initial, dfinal))
    B, T, C = x.shape
    W = w.shape[1]
    spans = [(b, 0, T) for b in range(B)] if cu is None else \
        [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]
    dx, dw, db = np.zeros_like(x), np.zeros_like(w), np.zeros(C)
    dinit = np.zeros((len(spans), W - 1, C))
    for n, (b, bos, eos) in enumerate(spans):
        first = np.zeros((W - 1, C)) if initial is None else initial[n]
        ext = np.concatenate([first, x[b, bos:eos]])
        dext = np.zeros_like(ext)
        L = eos - bos
        if dfinal is not None:
            dext[L:] += dfinal[n]
        for t in range(L):
            u = (0.0 if bias is None else bias) + (w.T * ext[t:t + W]).sum(0)
            s = sigmoid(u)
            du = dy[b, bos + t] * (s * (1.0 + u * (1.0 - s)) if silu else 1.0)
            dext[t:t + W] += w.T * du
            dw += (ext[t:t + W] * du).T
            db += du
        dinit[n], dx[b, bos:eos] = dext[:W - 1], dext[W - 1:]
    return dx, dw, db, dinit
