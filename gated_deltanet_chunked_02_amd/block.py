"""Binding of libgdn's block norm: argument checks and marshalling only.

    x, y, post_rstd, rstd = block_norm(x, h=None, weight=None, post_norm=False, post_weight=None,
                                       gate=None, activation=None, scale=None,
                                       residual_scale=1.0, pre_norm=True, eps=1e-5)
    dx, dh, dgate, dweight, dpost_weight, dscale = block_norm_bwd(dy, dx, x, h, post_rstd, rstd,
                                                                  ...)
"""
from __future__ import annotations

import ctypes

import torch
from torch import Tensor

from . import _MOST, ACTIVATIONS, GdnError, _fits, _launch, load
from .ssm import _CODES, _addresses, _f32, _new, _on, _rows, _stream, _workspace


class GdnBlockNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("post_norm", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("h_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


def declare(lib):
    """Argument types of the calls this module makes (run once, when the library is loaded)."""
    P, D = ctypes.c_void_p, ctypes.POINTER(GdnBlockNormDesc)
    lib.gdn_block_norm_bwd_workspace_size.restype = ctypes.c_size_t
    lib.gdn_block_norm_bwd_workspace_size.argtypes = [D, ctypes.POINTER(ctypes.c_int)]
    lib.gdn_block_norm_fwd.restype = ctypes.c_int
    lib.gdn_block_norm_fwd.argtypes = [D] + [P] * 11
    lib.gdn_block_norm_bwd.restype = ctypes.c_int
    lib.gdn_block_norm_bwd.argtypes = [D] + [P] * 17


def gdn_block_norm_fwd(desc, x, h, gate, post_weight, scale, weight, x_out, y, post_rstd, rstd,
                       stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_block_norm_fwd(
        ctypes.byref(desc), *_addresses((x, h, gate, post_weight, scale, weight, x_out, y,
                                        post_rstd, rstd)), _stream(stream)))


def gdn_block_norm_bwd_workspace_size(desc: GdnBlockNormDesc) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_block_norm_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_block_norm_bwd_workspace_size")
    return int(n)


def gdn_block_norm_bwd(desc, x, h, gate, post_weight, scale, weight, post_rstd, rstd, dx_out, dy,
                       dx, dh, dgate, dpost_weight, dscale, dweight, stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_block_norm_bwd(
        ctypes.byref(desc), *_addresses((x, h, gate, post_weight, scale, weight, post_rstd, rstd,
                                        dx_out, dy, dx, dh, dgate, dpost_weight, dscale,
                                        dweight)), _stream(stream)))


def _spaced(t):
    """(t, elements from one row of channels to the next), rows one after another as 0; a copy of a
    tensor whose rows are not evenly spaced."""
    if t is None or t.is_contiguous():
        return t, 0
    return _rows(t.flatten(0, -2) if t.dim() > 2 else t, 1)


def _block_operands(x, h, weight, post_norm, post_weight, gate, activation, scale, residual_scale,
                    eps, dtype):
    if not isinstance(x, Tensor):
        raise TypeError("x must be a torch tensor")
    code, shape = _CODES.get(x.dtype), x.shape
    if code is None:
        raise TypeError("x must be bf16 or fp32, got %s" % x.dtype)
    if len(shape) < 2 or shape[-1] == 0:
        raise ValueError("x must be [..., channels]")
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be None, 'none' or 'silu'")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    if h is None:
        if gate is not None or post_weight is not None or scale is not None or post_norm:
            raise ValueError("gate, post_norm, post_weight and scale belong to h")
        dtype = x.dtype if dtype is None else dtype
    else:
        if not isinstance(h, Tensor) or (dtype is not None and h.dtype != dtype):
            raise TypeError("h must be a torch tensor%s" % (" of %s" % dtype if dtype else ""))
        dtype = h.dtype
    if dtype not in _CODES or (dtype == torch.float32 and x.dtype != torch.float32):
        raise TypeError("h and y must have x's dtype, or be bf16 beside an fp32 x (got %s, %s)"
                        % (dtype, x.dtype))
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight belongs to post_norm")
    for name, t in (("h", h), ("gate", gate)):
        if t is None:
            continue
        if not isinstance(t, Tensor) or t.dtype != dtype:
            raise TypeError("%s must be a tensor of dtype %s" % (name, dtype))
        if t.shape != shape:
            raise ValueError("%s must have x's shape %s, got %s" % (name, list(shape),
                                                                    list(t.shape)))
    C = shape[-1]
    rows = x.numel() // C
    if not 0 < x.numel() <= _MOST:
        _fits(rows, C)
    params = (_f32("post_weight", post_weight, (C,)), _f32("scale", scale, (C,)),
              _f32("weight", weight, (C,)))
    h, sh = _spaced(h)
    gate, sg = _spaced(gate)
    desc = GdnBlockNormDesc(rows, C, _CODES[dtype], code, int(bool(post_norm)),
                            ACTIVATIONS[activation], eps, residual_scale, sh, sg, None, 0)
    return desc, dtype, x.contiguous(), h, gate, params


def block_norm(x, h=None, weight=None, post_norm=False, post_weight=None, gate=None,
               activation=None, scale=None, residual_scale=1.0, pre_norm=True, eps=1e-5,
               dtype=None, inplace=False):
    """A block's output h added to the residual stream x, and the next block's input y, on the
    current stream: z = norm(h) post_weight act(gate), x' = x + residual_scale scale z,
    y = norm(x') weight (RMS norms over the last axis).

    x: [..., channels], bf16 or fp32; h, gate: x's shape, x's dtype or bf16 beside an fp32 x (h
    None: x' is x, y its norm, of dtype ``dtype``); weight, post_weight, scale: [channels] fp32 or
    None (ones).  post_norm: whether h is normed; pre_norm: whether y is made; ``inplace``: x' is
    written to x, which must be contiguous.  Returns (x', y, post_rstd, rstd): y of h's dtype or
    None, the norms' factors fp32 of x's leading shape, or None."""
    desc, dtype, xc, h, gate, (post_weight, scale, weight) = _block_operands(
        x, h, weight, post_norm, post_weight, gate, activation, scale, residual_scale, eps, dtype)
    if h is None and not pre_norm:
        raise ValueError("without h and pre_norm there is nothing to do")
    if weight is not None and not pre_norm:
        raise ValueError("weight belongs to pre_norm")
    if inplace and xc is not x:
        raise ValueError("x must be contiguous to be written in place")
    dev = x.device
    _on(dev, x=x, h=h, gate=gate, weight=weight, post_weight=post_weight, scale=scale)
    lead = x.shape[:-1]
    out = xc if inplace or h is None else _new(xc)
    y = torch.empty_like(xc, dtype=dtype) if pre_norm else None
    post_rstd = xc.new_empty(lead, dtype=torch.float32) if post_norm else None
    rstd = xc.new_empty(lead, dtype=torch.float32) if pre_norm else None
    st = _launch(dev, gdn_block_norm_fwd, desc, xc, h, gate, post_weight, scale, weight,
                 None if h is None else out, y, post_rstd, rstd)
    if st != 0:
        raise GdnError(st, "gdn_block_norm_fwd")
    return out, y, post_rstd, rstd


def block_norm_bwd(dy, dx, x, h=None, post_rstd=None, rstd=None, weight=None, post_norm=False,
                   post_weight=None, gate=None, activation=None, scale=None, residual_scale=1.0,
                   workspace=None):
    """Gradients of block_norm's inputs on the current stream, given the gradients ``dy`` of y (None
    where it was left out) and ``dx`` of x' (None: zero), one of them at least, the forward's inputs
    (x as it was before) and its two factors.  Returns (dx, dh, dgate, dweight, dpost_weight,
    dscale): dx in x's dtype, dh and dgate in h's, the others [channels] fp32; None where the input
    is None (of the weights too)."""
    if dy is None and dx is None:
        raise TypeError("dy or dx is required")
    desc, dtype, x, h, gate, (post_weight, scale, weight) = _block_operands(
        x, h, weight, post_norm, post_weight, gate, activation, scale, residual_scale, 0.0,
        dy.dtype if h is None and isinstance(dy, Tensor) else None)
    for name, t, want in (("dy", dy, dtype), ("dx", dx, x.dtype)):
        if t is None:
            continue
        if not isinstance(t, Tensor) or t.dtype != want:
            raise TypeError("%s must be a tensor of dtype %s" % (name, want))
        if t.shape != x.shape:
            raise ValueError("%s must have x's shape %s, got %s" % (name, list(x.shape),
                                                                    list(t.shape)))
    if (dy is not None and rstd is None) or (post_norm and post_rstd is None):
        raise TypeError("the forward's rstd (with dy) and post_rstd (with post_norm) are required")
    lead = x.shape[:-1]
    rstd, post_rstd = _f32("rstd", rstd, lead), _f32("post_rstd", post_rstd, lead)
    if weight is not None and dy is None:
        raise ValueError("weight belongs to dy")
    dev = x.device
    _on(dev, x=x, h=h, gate=gate, dy=dy, dx=dx, weight=weight, post_weight=post_weight,
        scale=scale, rstd=rstd, post_rstd=post_rstd, workspace=workspace)
    dy = None if dy is None else dy.contiguous()
    dx = None if dx is None else dx.contiguous()
    like = lambda t: None if t is None else torch.empty_like(x, dtype=dtype)  # noqa: E731
    out, dh, dgate = _new(x), like(h), like(gate)
    dpost, dscale, dweight = map(_new, (post_weight, scale, weight))
    ws = _workspace(desc, gdn_block_norm_bwd_workspace_size(desc), workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_block_norm_bwd, desc, x, h, gate, post_weight, scale, weight, post_rstd,
                 rstd, dx, dy, out, dh, dgate, dpost, dscale, dweight)
    if st != 0:
        raise GdnError(st, "gdn_block_norm_bwd")
    return out, dh, dgate, dweight, dpost, dscale
