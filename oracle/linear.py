"""Oracle for linear attention with a decay for each head — TEST INFRASTRUCTURE ONLY (the same import
rules as the rest of ``oracle/``).

Plain fp64 numpy from the definition, token by token, with q/k head hk(h) = h / (H / Hg):

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t

and the derivative of sum(o do) + sum(ht dht) by going back through the tokens, dS the gradient of
S_t (dS after the last token: dht):

    dS += scale q_t do_t^T
    dq_t = scale S_t do_t,  dk_t = dS v_t,  dv_t = dS^T k_t,  dg_t = exp(g_t) <dS, S_{t-1}>
    dS <- exp(g_t) dS       (after the first token: dh0)
"""
from __future__ import annotations

import numpy as np

from .selective import _spans


def _decays(g, B, T, H):
    g = np.asarray(g, np.float64)
    return np.exp(np.broadcast_to(g, (B, T, H)) if g.ndim == 1 else g)


def attention(q, k, v, g, scale, h0=None, cu=None):
    """(o, ht) in fp64."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, T, Hg, Dk = q.shape
    H, Dv = v.shape[2:]
    keep = _decays(g, B, T, H)
    rep = H // Hg
    spans = _spans(q, cu)
    o, ht = np.zeros((B, T, H, Dv)), np.zeros((len(spans), H, Dk, Dv))
    for n, (b, bos, eos) in enumerate(spans):
        S = np.zeros((H, Dk, Dv)) if h0 is None else np.array(h0[n], np.float64)
        for t in range(bos, eos):
            kt, qt = np.repeat(k[b, t], rep, 0), np.repeat(q[b, t], rep, 0)
            S = keep[b, t][:, None, None] * S + kt[:, :, None] * v[b, t][:, None, :]
            o[b, t] = scale * (qt[:, :, None] * S).sum(1)
        ht[n] = S
    return o, ht


def attention_backward(q, k, v, g, do, scale, h0=None, dht=None, cu=None):
    """Gradients in fp64, as a dict: dq, dk, dv, dg, dh0 (tokens that no sequence has keep zeros)."""
    head = np.asarray(g).ndim == 1
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    B, T, Hg, Dk = q.shape
    H, Dv = v.shape[2:]
    keep = _decays(g, B, T, H)
    rep = H // Hg
    spans = _spans(q, cu)
    out = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v),
               dg=np.zeros((B, T, H)), dh0=np.zeros((len(spans), H, Dk, Dv)))
    for n, (b, bos, eos) in enumerate(spans):
        states = [np.zeros((H, Dk, Dv)) if h0 is None else np.array(h0[n], np.float64)]
        for t in range(bos, eos):
            states.append(keep[b, t][:, None, None] * states[-1] +
                          np.repeat(k[b, t], rep, 0)[:, :, None] * v[b, t][:, None, :])
        dS = np.zeros((H, Dk, Dv)) if dht is None else np.array(dht[n], np.float64)
        for t in range(eos - 1, bos - 1, -1):
            S, before = states[t - bos + 1], states[t - bos]
            kt, qt = np.repeat(k[b, t], rep, 0), np.repeat(q[b, t], rep, 0)
            dS = dS + scale * qt[:, :, None] * do[b, t][:, None, :]
            dq = scale * (S * do[b, t][:, None, :]).sum(2)
            dk = (dS * v[b, t][:, None, :]).sum(2)
            out["dq"][b, t] = dq.reshape(Hg, rep, Dk).sum(1)
            out["dk"][b, t] = dk.reshape(Hg, rep, Dk).sum(1)
            out["dv"][b, t] = (dS * kt[:, :, None]).sum(1)
            out["dg"][b, t] = keep[b, t] * (dS * before).sum((1, 2))
            dS = keep[b, t][:, None, None] * dS
        out["dh0"][n] = dS
    if head:
        out["dg"] = out["dg"].sum((0, 1))
    return out
