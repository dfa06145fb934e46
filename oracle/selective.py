"""Oracle for the selective state-space scan — TEST INFRASTRUCTURE ONLY (the same import rules
as the rest of ``oracle/``).

Plain fp64 numpy from the definition, token by token: with group g(c) = c // (C / G) and
step_t = softplus(dt_t + bias) (or dt_t + bias),

    h_t[c, s] = exp(step_t[c] A[c, s]) h_{t-1}[c, s] + step_t[c] x_t[c] B_t[g(c), s]
    y_t[c]    = (sum_s C_t[g(c), s] h_t[c, s] + D[c] x_t[c]) silu(z_t[c])

and the derivative of sum(y dy) + sum(ht dht) by going back through the tokens:

    e_t = dy_t silu(z_t),   g_t = e_t C_t + exp(step_{t+1} A) g_{t+1}    (g after the last: dht)
    q_t = g_t exp(step_t A) h_{t-1}
    dA += step_t q_t        dstep_t = sum_s (A q_t + x_t B_t g_t)     ddt = dstep step'(.)
    dx_t = step_t sum_s B_t g_t + D e_t        dD += x_t e_t          dbias += ddt_t
    dB_t[g, s] = sum over the group's c of step_t x_t g_t             dC_t[g, s] = sum of e_t h_t
    dz_t = dy_t (sum_s C_t h_t + D x_t) silu'(z_t)                    dh0 = exp(step_1 A) g_1
"""
from __future__ import annotations

import numpy as np


def softplus(v):
    return np.logaddexp(0.0, v)


def sigmoid(v):
    return np.exp(-np.logaddexp(0.0, -np.asarray(v, np.float64)))


def silu(v):
    return v * sigmoid(v)


def _spans(x, cu):
    """(batch row, first token, end) of every sequence."""
    B, T = x.shape[:2]
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]


def _wide(m, C):
    """[G, S] -> [C, S]: each group's row for its channels."""
    return np.repeat(m, C // m.shape[0], axis=0)


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False, h0=None, cu=None):
    """(y, ht) in fp64."""
    f = lambda t: None if t is None else np.asarray(t, np.float64)  # noqa: E731
    x, dt, A, B, C, D, z, dt_bias, h0 = map(f, (x, dt, A, B, C, D, z, dt_bias, h0))
    ch, S = A.shape
    spans = _spans(x, cu)
    y = np.zeros_like(x)
    ht = np.zeros((len(spans), ch, S))
    step = dt if dt_bias is None else dt + dt_bias
    step = softplus(step) if dt_softplus else step
    for n, (b, bos, eos) in enumerate(spans):
        h = np.zeros((ch, S)) if h0 is None else h0[n].copy()
        for t in range(bos, eos):
            d = step[b, t][:, None]
            h = np.exp(d * A) * h + d * x[b, t][:, None] * _wide(B[b, t], ch)
            y[b, t] = (h * _wide(C[b, t], ch)).sum(1)
        ht[n] = h
    if D is not None:
        y += D * x
    if z is not None:
        y *= silu(z)
    return y, ht


def scan_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, dt_softplus=False, h0=None,
                  dht=None, cu=None):
    """Gradients in fp64, as a dict: dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 (tokens that no
    sequence has keep zeros)."""
    f = lambda t: None if t is None else np.asarray(t, np.float64)  # noqa: E731
    x, dt, A, B, C, dy, D, z, dt_bias, h0, dht = map(
        f, (x, dt, A, B, C, dy, D, z, dt_bias, h0, dht))
    ch, S = A.shape
    G = B.shape[2]
    per = ch // G
    spans = _spans(x, cu)
    raw = dt if dt_bias is None else dt + dt_bias
    step = softplus(raw) if dt_softplus else raw
    slope = sigmoid(raw) if dt_softplus else np.ones_like(raw)
    gate = np.ones_like(x) if z is None else silu(z)
    dgate = None if z is None else sigmoid(z) * (1.0 + z * (1.0 - sigmoid(z)))
    Dv = np.zeros(ch) if D is None else D
    out = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dA=np.zeros_like(A),
               dB=np.zeros_like(B), dC=np.zeros_like(C), dD=np.zeros(ch),
               dz=np.zeros_like(x), dbias=np.zeros(ch), dh0=np.zeros((len(spans), ch, S)))
    for n, (b, bos, eos) in enumerate(spans):
        hs = [np.zeros((ch, S)) if h0 is None else h0[n]]
        for t in range(bos, eos):
            d = step[b, t][:, None]
            hs.append(np.exp(d * A) * hs[-1] + d * x[b, t][:, None] * _wide(B[b, t], ch))
        g = np.zeros((ch, S)) if dht is None else dht[n].copy()
        for t in range(eos - 1, bos - 1, -1):
            h, before = hs[t - bos + 1], hs[t - bos]
            Bt, Ct = _wide(B[b, t], ch), _wide(C[b, t], ch)
            d, e = step[b, t], dy[b, t] * gate[b, t]
            if z is not None:
                out["dz"][b, t] = dy[b, t] * ((h * Ct).sum(1) + Dv * x[b, t]) * dgate[b, t]
            g = g + e[:, None] * Ct
            a = np.exp(d[:, None] * A)
            q = g * a * before
            out["dA"] += d[:, None] * q
            gB = (g * Bt).sum(1)
            ddt = ((A * q).sum(1) + x[b, t] * gB) * slope[b, t]
            out["ddt"][b, t] = ddt
            out["dbias"] += ddt
            out["dx"][b, t] = d * gB + Dv * e
            out["dD"] += x[b, t] * e
            out["dB"][b, t] = (g * (d * x[b, t])[:, None]).reshape(G, per, S).sum(1)
            out["dC"][b, t] = (h * e[:, None]).reshape(G, per, S).sum(1)
            g = a * g
        out["dh0"][n] = g
    return out
