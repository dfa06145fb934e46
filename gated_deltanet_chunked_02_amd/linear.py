"""Binding of libgdn's linear attention calls: argument checks and marshalling only.

    o, ht = linear_attention(q, k, v, g, scale=None, initial_state=None,
                             output_final_state=True, cu_seqlens=None)
    dq, dk, dv, dg, dh0 = linear_attention_bwd(q, k, v, g, do, dht=None, ...)
    o = linear_state_update(state, q, k, v, g, cache_indices=None, out_indices=None)

Tensors whose token rows are contiguous, evenly spaced and aligned to 16 bytes (the slices of a
projection's last axis, usually) are passed as they are; others are copied first.
"""
from __future__ import annotations

import ctypes

import torch
from torch import Tensor

from . import _MOST, GdnError, _fits, _launch, _need, load
from .ssm import (_CODES, _addresses, _f32, _indices, _new, _on, _rows, _sequences, _stream,
                  _workspace)


class GdnLinearDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("N", ctypes.c_int32),
                ("H", ctypes.c_int32), ("Hg", ctypes.c_int32), ("Dk", ctypes.c_int32),
                ("Dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("head_decay", ctypes.c_int32), ("state_lines", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


def declare(lib):
    """Argument types of the calls this module makes (run once, when the library is loaded)."""
    P, S = ctypes.c_void_p, ctypes.c_size_t
    D, st = ctypes.POINTER(GdnLinearDesc), ctypes.POINTER(ctypes.c_int)
    for name in ("gdn_linear_attn_workspace_size", "gdn_linear_attn_bwd_workspace_size"):
        getattr(lib, name).restype = S
        getattr(lib, name).argtypes = [D, st]
    for name, pointers in (("gdn_linear_attn_fwd", 9), ("gdn_linear_attn_bwd", 14),
                           ("gdn_linear_state_update", 9)):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = [D] + [P] * pointers


def gdn_linear_attn_workspace_size(desc: GdnLinearDesc) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_linear_attn_workspace_size(ctypes.byref(desc), ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_linear_attn_workspace_size")
    return int(n)


def gdn_linear_attn_bwd_workspace_size(desc: GdnLinearDesc) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_linear_attn_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_linear_attn_bwd_workspace_size")
    return int(n)


def gdn_linear_attn_fwd(desc, q, k, v, g, h0, cu_seqlens, o, ht, stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_linear_attn_fwd(
        ctypes.byref(desc), *_addresses((q, k, v, g, h0, cu_seqlens, o, ht)), _stream(stream)))


def gdn_linear_attn_bwd(desc, q, k, v, g, h0, cu_seqlens, do, dht, dq, dk, dv, dg, dh0,
                        stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_linear_attn_bwd(
        ctypes.byref(desc), *_addresses((q, k, v, g, h0, cu_seqlens, do, dht, dq, dk, dv, dg,
                                        dh0)), _stream(stream)))


def gdn_linear_state_update(desc, state, q, k, v, g, cache_indices, out_indices, o,
                            stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_linear_state_update(
        ctypes.byref(desc), *_addresses((state, q, k, v, g, cache_indices, out_indices, o)),
        _stream(stream)))


def _aligned(t):
    """t, or a copy of it at an address of 16 bytes."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _aligned_rows(t, lead):
    """_rows, for rows that the kernels read 16 bytes at a time."""
    t, row = _rows(t, lead)
    if row and (row * t.element_size() % 16 or t.data_ptr() % 16 or row >= 1 << 23):
        t, row = t.contiguous(), 0
    return (t, row) if row else (_aligned(t), 0)


def _linear_operands(q, k, v, g, scale, lead):
    """Checks of the operands that prompts and single tokens share, and the descriptor but for the
    batch's shape.  ``lead``: axes before the heads."""
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        if not isinstance(t, Tensor):
            raise TypeError("%s must be a torch tensor" % name)
    shape, wide = q.shape, v.shape
    axes = "B, T" if lead == 2 else "B"
    if len(shape) != lead + 2 or k.shape != shape:
        raise ValueError("q and k must be [%s, q/k heads, Dk], got %s and %s"
                         % (axes, list(shape), list(k.shape)))
    code = _CODES.get(q.dtype)
    if code is None:
        raise TypeError("q must be bf16 or fp32, got %s" % q.dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype (got %s, %s, %s)"
                        % (q.dtype, k.dtype, v.dtype))
    if len(wide) != lead + 2 or wide[:lead] != shape[:lead]:
        raise ValueError("v must be [%s, heads, Dv] with q's %s, got %s" % (axes, axes, list(wide)))
    Hg, Dk = shape[lead:]
    H, Dv = wide[lead:]
    if min(Hg, Dk, H, Dv) == 0 or H % Hg:
        raise ValueError("v heads (%d) must be a multiple of q/k heads (%d), and no size 0"
                         % (H, Hg))
    if g.dtype != torch.float32:
        raise TypeError("g must be fp32, got %s" % g.dtype)
    head = g.dim() == 1
    if g.shape != ((H,) if head else wide[:lead + 1]):
        raise ValueError("g must be [%d] or %s, got %s"
                         % (H, list(wide[:lead + 1]), list(g.shape)))
    if not 0 < max(q.numel(), v.numel()) <= _MOST:  # else no axis is longer either
        _fits(*shape, *wide)
    q, sq = _aligned_rows(q, lead)
    k, sk = _aligned_rows(k, lead)
    v, sv = _aligned_rows(v, lead)
    # B, T, N and state_lines are the caller's
    desc = GdnLinearDesc(0, 0, 0, H, Hg, Dk, Dv, code, int(head), 0,
                         Dk ** -0.5 if scale is None else scale, sq, sk, sv, None, 0)
    return desc, q, k, v, g.contiguous()


def linear_attention(q, k, v, g, scale=None, initial_state=None, output_final_state=True,
                     cu_seqlens=None, workspace=None):
    """Linear attention with a decay for each head on the current stream:
    S = exp(g) S + k v^T, o = scale S^T q.

    q, k: [B, T, q/k heads, Dk]; v: [B, T, heads, Dv] (bf16 or fp32); g: [heads] or [B, T, heads]
    fp32, the log-decay; scale: Dk^-0.5 by default; initial_state [N, heads, Dk, Dv] fp32 or None;
    cu_seqlens [N + 1] for a packed batch (B == 1; o of tokens that no sequence has is not written).
    Dk and Dv are multiples of 8 up to 256.  Returns (o [B, T, heads, Dv] in q's dtype, final state
    fp32 or None)."""
    desc, q, k, v, g = _linear_operands(q, k, v, g, scale, 2)
    cu, N = _sequences(q, cu_seqlens)
    states = (N, desc.H, desc.Dk, desc.Dv)
    h0 = _aligned(_f32("initial_state", initial_state, states))
    dev = q.device
    _on(dev, q=q, k=k, v=v, g=g, initial_state=h0, cu_seqlens=cu, workspace=workspace)
    desc.B, desc.T, desc.N = q.shape[0], q.shape[1], N
    o = _new(v)
    ht = None
    if output_final_state:
        ht = g.new_empty(states) if h0 is None else _new(h0)
    if q.shape[0] == 0:
        return o, ht
    ws = _workspace(desc, gdn_linear_attn_workspace_size(desc), workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_linear_attn_fwd, desc, q, k, v, g, h0, cu, o, ht)
    if st != 0:
        raise GdnError(st, "gdn_linear_attn_fwd")
    return o, ht


def linear_attention_bwd(q, k, v, g, do, dht=None, scale=None, initial_state=None,
                         cu_seqlens=None, need_dg=True, workspace=None):
    """Gradients of linear_attention's inputs on the current stream, given the gradient ``do`` of o
    (v's shape and dtype) and ``dht`` of the final state (fp32, or None: zero); the forward's inputs
    as there, Dk and Dv up to 128.  Returns (dq, dk, dv, dg, dinitial_state): dq, dk, dv in q's
    dtype, dg (g's shape; None without ``need_dg``) and dinitial_state (None where the input is None)
    in fp32.  Those of tokens of a packed batch that no sequence has are not written.  The workspace
    is larger than the inputs (see include/gdn.h); one may be given (uint8)."""
    desc, q, k, v, g = _linear_operands(q, k, v, g, scale, 2)
    cu, N = _sequences(q, cu_seqlens)
    states = (N, desc.H, desc.Dk, desc.Dv)
    h0 = _aligned(_f32("initial_state", initial_state, states))
    dht = _aligned(_f32("dht", dht, states))
    _need(isinstance(do, Tensor) and do.dtype == v.dtype, TypeError,
          "do must be a tensor of v's dtype %s" % v.dtype)
    _need(do.shape == v.shape, ValueError, "do must have v's shape %s, got %s"
          % (list(v.shape), list(do.shape)))
    dev = q.device
    _on(dev, q=q, k=k, v=v, g=g, do=do, initial_state=h0, dht=dht, cu_seqlens=cu,
        workspace=workspace)
    do = _aligned(do.contiguous())
    desc.B, desc.T, desc.N = q.shape[0], q.shape[1], N
    dq, dk, dv, dh0 = map(_new, (q, k, v, h0))
    dg = _new(g) if need_dg else None
    if q.shape[0] == 0:
        return dq, dk, dv, dg if dg is None else dg.zero_(), dh0
    need = gdn_linear_attn_bwd_workspace_size(desc)
    ws = _workspace(desc, need, workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_linear_attn_bwd, desc, q, k, v, g, h0, cu, do, dht, dq, dk, dv, dg, dh0)
    if st != 0:
        raise GdnError(st, "gdn_linear_attn_bwd")
    return dq, dk, dv, dg, dh0


def linear_state_update(state, q, k, v, g, scale=None, cache_indices=None, out_indices=None):
    """One token of each sequence: linear attention's step on the current stream.

    state: [lines, heads, Dk, Dv] fp32, contiguous, updated in place; q, k: [B, q/k heads, Dk]; v:
    [B, heads, Dv]; g: [heads] or [B, heads] fp32.  Sequence b reads line cache_indices[b] (b when
    None) and writes line out_indices[b] (the line it read when None).  Returns o [B, heads, Dv] in
    q's dtype."""
    desc, q, k, v, g = _linear_operands(q, k, v, g, scale, 1)
    n = q.shape[0]
    if not isinstance(state, Tensor) or state.dtype != torch.float32 or \
            not state.is_contiguous() or state.data_ptr() % 16:
        raise TypeError("state must be a contiguous fp32 tensor aligned to 16 bytes")
    if state.dim() != 4 or state.shape[0] == 0 or \
            state.shape[1:] != (desc.H, desc.Dk, desc.Dv):
        raise ValueError("state must be [lines, %d, %d, %d], got %s"
                         % (desc.H, desc.Dk, desc.Dv, list(state.shape)))
    read, write = _indices("cache_indices", cache_indices, n), _indices("out_indices",
                                                                        out_indices, n)
    _need(read is not None or state.shape[0] >= n, ValueError,
          "state has fewer lines (%d) than there are sequences (%d)" % (state.shape[0], n))
    if state.shape[0] > _MOST:
        _fits(state.shape[0])
    dev = q.device
    _on(dev, state=state, q=q, k=k, v=v, g=g, cache_indices=read, out_indices=write)
    o = _new(v)
    if n == 0:
        return o
    desc.B, desc.T, desc.N, desc.state_lines = n, 1, n, state.shape[0]
    st = _launch(dev, gdn_linear_state_update, desc, state, q, k, v, g, read, write, o)
    if st != 0:
        raise GdnError(st, "gdn_linear_state_update")
    return o
