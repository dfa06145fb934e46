"""Binding of libgdn's calls for a selective state-space layer: argument checks and marshalling
only.

    y, ht = selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                           initial_state=None, output_final_state=True, cu_seqlens=None)
    dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0 = selective_scan_bwd(x, dt, A, B, C, dy, ...)
    y = selective_state_update(state, x, dt, A, B, C, ..., cache_indices=None,
                               out_indices=None)
    dx, dweight, dbias, dinitial = causal_conv1d_bwd(x, weight, dy, bias=None, ...)
    y, mean, rstd = group_norm(x, num_groups, weight=None, bias=None, eps=1e-5,
                               activation=None, gate=None)
    dx, dweight, dbias, dgate = group_norm_bwd(dy, x, num_groups, mean, rstd, ...)

Tensors whose token rows are contiguous and evenly spaced (a slice of a projection's last axis)
are passed as they are; others are copied first.
"""
from __future__ import annotations

import ctypes

import torch
from torch import Tensor

from . import (_MOST, ACTIVATIONS, BF16, F32, GdnConvDesc, GdnError, _check_devices,
               _current_stream, _fits, _launch, _need, _validate_conv, load)

_CODES = {torch.bfloat16: BF16, torch.float32: F32}


class GdnScanDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("N", ctypes.c_int32),
                ("channels", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("dt_softplus", ctypes.c_int32), ("state_lines", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("z_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("c_stride", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class GdnNormDesc(ctypes.Structure):
    _fields_ = [("samples", ctypes.c_int32), ("positions", ctypes.c_int32),
                ("channels", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("eps", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


def declare(lib):
    """Argument types of the calls this module makes (run once, when the library is loaded)."""
    P, S = ctypes.c_void_p, ctypes.c_size_t
    D, st = ctypes.POINTER(GdnScanDesc), ctypes.POINTER(ctypes.c_int)
    lib.gdn_selective_scan_workspace_size.restype = S
    lib.gdn_selective_scan_workspace_size.argtypes = [D, st]
    lib.gdn_selective_scan_fwd.restype = ctypes.c_int
    lib.gdn_selective_scan_fwd.argtypes = [D] + [P] * 13
    lib.gdn_selective_scan_bwd_workspace_size.restype = S
    lib.gdn_selective_scan_bwd_workspace_size.argtypes = [D, st]
    lib.gdn_selective_scan_bwd.restype = ctypes.c_int
    lib.gdn_selective_scan_bwd.argtypes = [D] + [P] * 22
    lib.gdn_selective_state_update.restype = ctypes.c_int
    lib.gdn_selective_state_update.argtypes = [D] + [P] * 13
    V = ctypes.POINTER(GdnConvDesc)
    lib.gdn_causal_conv1d_bwd_workspace_size.restype = S
    lib.gdn_causal_conv1d_bwd_workspace_size.argtypes = [V, st]
    lib.gdn_causal_conv1d_bwd.restype = ctypes.c_int
    lib.gdn_causal_conv1d_bwd.argtypes = [V] + [P] * 12 + [S, P]
    M = ctypes.POINTER(GdnNormDesc)
    lib.gdn_group_norm_workspace_size.restype = S
    lib.gdn_group_norm_workspace_size.argtypes = [M, ctypes.c_int32, st]
    lib.gdn_group_norm_fwd.restype = ctypes.c_int
    lib.gdn_group_norm_fwd.argtypes = [M] + [P] * 8
    lib.gdn_group_norm_bwd.restype = ctypes.c_int
    lib.gdn_group_norm_bwd.argtypes = [M] + [P] * 12


def _stream(stream):
    if type(stream) is int:
        return stream
    if stream is None:
        return _current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _addresses(tensors):
    return [t if t is None or type(t) is int else t.data_ptr() for t in tensors]


def gdn_selective_scan_workspace_size(desc: GdnScanDesc) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_selective_scan_workspace_size(ctypes.byref(desc), ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_selective_scan_workspace_size")
    return int(n)


def gdn_selective_scan_fwd(desc, x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, y, ht,
                           stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_selective_scan_fwd(
        ctypes.byref(desc), *_addresses((x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, y, ht)),
        _stream(stream)))


def gdn_selective_scan_bwd_workspace_size(desc: GdnScanDesc) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_selective_scan_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_selective_scan_bwd_workspace_size")
    return int(n)


def gdn_selective_scan_bwd(desc, x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dy, dht, dx, ddt,
                           dA, dB, dC, dD, dz, ddt_bias, dh0, stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_selective_scan_bwd(
        ctypes.byref(desc), *_addresses((x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, dy, dht,
                                        dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)),
        _stream(stream)))


def gdn_selective_state_update(desc, state, x, dt, A, B, C, D, z, dt_bias, cache_indices,
                               out_indices, y, stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_selective_state_update(
        ctypes.byref(desc), *_addresses((state, x, dt, A, B, C, D, z, dt_bias, cache_indices,
                                        out_indices, y)), _stream(stream)))


def _code(t):
    """The library's code of a tensor's dtype, or None."""
    return _CODES.get(t.dtype)


def _rows(t, lead):
    """(t, elements from one row to the next) for a tensor [*lead, ...] whose rows are
    contiguous and evenly spaced over its one or two leading axes; a contiguous copy of any
    other (0: rows one after another)."""
    if t.is_contiguous():
        return t, 0
    shape, stride = t.shape, t.stride()
    width = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        n = shape[i]
        if n != 1 and stride[i] != width:
            return t.contiguous(), 0
        width *= n
    if lead == 1:
        row = stride[0]
    elif shape[1] == 1:
        row = stride[0]
    else:
        row = stride[1]
        if shape[0] != 1 and stride[0] != row * shape[1]:
            return t.contiguous(), 0
    return (t, row) if row >= width else (t.contiguous(), 0)


def _new(t):
    """A new contiguous tensor of t's shape, dtype and device, or None.  t is contiguous or has
    evenly spaced rows (see _rows), whose order an empty_like keeps; it takes a third of the time of
    an empty with the three given."""
    return None if t is None else torch.empty_like(t)


def _on(device, **named):
    """Every tensor given on ``device``, a CUDA (HIP) device."""
    _check_devices(named, device)


def _f32(name, t, shape):
    if t is None:
        return None
    if not isinstance(t, Tensor) or t.dtype != torch.float32:
        raise TypeError("%s must be an fp32 tensor" % name)
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    return t.contiguous()


def _indices(name, t, n):
    if t is None:
        return None
    if not isinstance(t, Tensor) or t.dtype not in (torch.int32, torch.int64):
        raise TypeError("%s must be an int32 or int64 tensor" % name)
    if t.shape != (n,):
        raise ValueError("%s must be [%d]" % (name, n))
    if t.dtype == torch.int64:  # outside the pool either way, where a bare cast would wrap into it
        t = t.clamp(-1, _MOST).to(torch.int32)
    return t.contiguous()


def _like(name, t, x):
    """A tensor of x's shape and dtype, or None."""
    if t is None:
        return
    if not isinstance(t, Tensor) or t.dtype != x.dtype:
        raise TypeError("%s must be a tensor of x's dtype %s" % (name, x.dtype))
    if t.shape != x.shape:
        raise ValueError("%s must have x's shape %s, got %s" % (name, list(x.shape),
                                                                list(t.shape)))


def _operands(x, dt, A, B, C, D, z, dt_bias, lead):
    """Checks of the operands that the scan and its single-token form share, and the descriptor
    but for the batch's shape.  ``lead``: axes before the channels."""
    for name, t in (("x", x), ("dt", dt), ("A", A), ("B", B), ("C", C)):
        if not isinstance(t, Tensor):
            raise TypeError("%s must be a torch tensor" % name)
    shape, dtype = x.shape, x.dtype
    if len(shape) != lead + 1:
        raise ValueError("x must be %s" % ("[B, T, channels]" if lead == 2 else "[B, channels]"))
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("x must be bf16 or fp32, got %s" % dtype)
    ch = shape[-1]
    if ch == 0:
        raise ValueError("x must have channels")
    _like("dt", dt, x)
    _like("z", z, x)
    if A.dim() != 2 or A.shape[0] != ch or A.shape[1] == 0:
        raise ValueError("A must be [channels, dstate] with %d channels, got %s"
                         % (ch, list(A.shape)))
    S = A.shape[1]
    A = _f32("A", A, (ch, S))
    rows = B.shape
    for name, t in (("B", B), ("C", C)):
        if t.dtype != dtype:
            raise TypeError("%s must have x's dtype %s" % (name, dtype))
        if t.shape != rows or len(rows) != lead + 2 or rows[:lead] != shape[:lead] or \
                rows[-1] != S:
            raise ValueError("%s must be %s with dstate %d, got %s" % (
                name, "[B, T, groups, dstate]" if lead == 2 else "[B, groups, dstate]", S,
                list(t.shape)))
    G = rows[lead]
    if G == 0 or ch % G:
        raise ValueError("the channels (%d) must be a multiple of the groups (%d)" % (ch, G))
    if not 0 < x.numel() <= _MOST or S > _MOST:  # else no axis is longer either
        _fits(*rows, *shape)
    D, dt_bias = _f32("D", D, (ch,)), _f32("dt_bias", dt_bias, (ch,))
    x, sx = _rows(x, lead)
    dt, sdt = _rows(dt, lead)
    B, sb = _rows(B, lead)
    C, sc = _rows(C, lead)
    sz = 0
    if z is not None:
        z, sz = _rows(z, lead)
    # B, T, N, dt_softplus and state_lines are the caller's
    desc = GdnScanDesc(0, 0, 0, ch, G, S, code, 0, 0, sx, sdt, sz, sb, sc, None, 0)
    return desc, x, dt, A, B, C, D, z, dt_bias


def _sequences(x, cu_seqlens):
    """(cu_seqlens as int32 or None, number of sequences) of x [B, T, ...]."""
    if cu_seqlens is None:
        return None, x.shape[0]
    _need(isinstance(cu_seqlens, torch.Tensor) and
          cu_seqlens.dtype in (torch.int32, torch.int64), TypeError,
          "cu_seqlens must be an int32 or int64 tensor")
    _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, ValueError,
          "cu_seqlens must be 1-D [N + 1]")
    _need(x.shape[0] == 1, ValueError, "a packed batch (cu_seqlens) needs B == 1")
    _fits(cu_seqlens.numel())
    return cu_seqlens.to(torch.int32).contiguous(), cu_seqlens.numel() - 1


def _workspace(desc, need, workspace, device):
    """Points the descriptor at the caller's workspace, or at a new one; returns it."""
    if workspace is not None:
        _need(isinstance(workspace, torch.Tensor) and workspace.dtype == torch.uint8 and
              workspace.is_contiguous(), TypeError,
              "workspace must be a contiguous uint8 tensor")
    if need:
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(need, device=device, dtype=torch.uint8)
        desc.workspace = workspace.data_ptr()
        desc.workspace_bytes = workspace.numel()
    return workspace


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                   initial_state=None, output_final_state=True, cu_seqlens=None,
                   workspace=None):
    """The selective scan on the current stream: per channel c and state s,
    h = exp(step A) h + step x B, y = (sum_s C h + D x) silu(z), step = dt + dt_bias, through
    softplus when ``dt_softplus``.

    x, dt, z: [B, T, channels] (bf16 or fp32; z None: no gate); A [channels, dstate] fp32;
    B, C: [B, T, groups, dstate], shared by channels / groups channels each; D, dt_bias
    [channels] fp32 or None; initial_state [N, channels, dstate] fp32 or None; cu_seqlens
    [N + 1] for a packed batch (B == 1; y of tokens that no sequence has is not written).  Returns (y
    in x's dtype, final state fp32 or None)."""
    desc, x, dt, A, B, C, D, z, dt_bias = _operands(x, dt, A, B, C, D, z, dt_bias, 2)
    cu, N = _sequences(x, cu_seqlens)
    h0 = _f32("initial_state", initial_state, (N, desc.channels, desc.dstate))
    dev = x.device
    _on(dev, x=x, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, initial_state=h0,
        cu_seqlens=cu, workspace=workspace)
    desc.B, desc.T, desc.N, desc.dt_softplus = x.shape[0], x.shape[1], N, int(bool(dt_softplus))
    y = _new(x)
    ht = None
    if output_final_state:
        ht = A.new_empty((N, desc.channels, desc.dstate)) if h0 is None else _new(h0)
    if x.shape[0] == 0:
        return y, ht
    ws = _workspace(desc, gdn_selective_scan_workspace_size(desc), workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_selective_scan_fwd, desc, x, dt, A, B, C, D, z, dt_bias, h0, cu, y, ht)
    if st != 0:
        raise GdnError(st, "gdn_selective_scan_fwd")
    return y, ht


def selective_scan_bwd(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, dt_softplus=False,
                       initial_state=None, dht=None, cu_seqlens=None, workspace=None):
    """Gradients of selective_scan's inputs on the current stream, given the gradient ``dy`` of y
    (x's shape and dtype) and ``dht`` of the final state (fp32, or None: zero); the forward's
    inputs as there.  Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinitial_state): dx, ddt,
    dz, dB, dC in x's dtype, the others in fp32, None where the input is None.  Those of tokens of a
    packed batch that no sequence has are unspecified.  The workspace is larger than the inputs (see
    include/gdn.h); one may be given (uint8)."""
    desc, x, dt, A, B, C, D, z, dt_bias = _operands(x, dt, A, B, C, D, z, dt_bias, 2)
    cu, N = _sequences(x, cu_seqlens)
    states = (N, desc.channels, desc.dstate)
    h0, dht = _f32("initial_state", initial_state, states), _f32("dht", dht, states)
    _need(dy is not None, TypeError, "dy is required")
    _like("dy", dy, x)
    dev = x.device
    _on(dev, x=x, dt=dt, A=A, B=B, C=C, dy=dy, D=D, z=z, dt_bias=dt_bias, initial_state=h0,
        dht=dht, cu_seqlens=cu, workspace=workspace)
    dy = dy.contiguous()
    desc.B, desc.T, desc.N, desc.dt_softplus = x.shape[0], x.shape[1], N, int(bool(dt_softplus))
    dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = map(_new, (x, dt, A, B, C, D, z, dt_bias, h0))
    if x.shape[0] == 0:
        return dx, ddt, dA.zero_(), dB, dC, _zero(dD), dz, _zero(dbias), dh0
    need = gdn_selective_scan_bwd_workspace_size(desc)
    ws = _workspace(desc, need, workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_selective_scan_bwd, desc, x, dt, A, B, C, D, z, dt_bias, h0, cu, dy, dht,
                 dx, ddt, dA, dB, dC, dD, dz, dbias, dh0)
    if st != 0:
        raise GdnError(st, "gdn_selective_scan_bwd")
    return dx, ddt, dA, dB, dC, dD, dz, dbias, dh0


def _zero(t):
    return None if t is None else t.zero_()


def selective_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None,
                           dt_softplus=False, cache_indices=None, out_indices=None):
    """One token of each sequence: the selective scan's step on the current stream.

    state: [lines, channels, dstate] fp32, contiguous, updated in place; x, dt, z:
    [B, channels]; B, C: [B, groups, dstate]; the rest as for selective_scan.  Sequence b reads
    line cache_indices[b] (b when None) and writes line out_indices[b] (the line it read when
    None).  Returns y [B, channels] in x's dtype."""
    desc, x, dt, A, B, C, D, z, dt_bias = _operands(x, dt, A, B, C, D, z, dt_bias, 1)
    n = x.shape[0]
    if not isinstance(state, Tensor) or state.dtype != torch.float32 or \
            not state.is_contiguous():
        raise TypeError("state must be a contiguous fp32 tensor")
    if state.dim() != 3 or state.shape[0] == 0 or state.shape[1:] != A.shape:
        raise ValueError("state must be [lines, %d, %d], got %s"
                         % (desc.channels, desc.dstate, list(state.shape)))
    read, write = _indices("cache_indices", cache_indices, n), _indices("out_indices",
                                                                        out_indices, n)
    _need(read is not None or state.shape[0] >= n, ValueError,
          "state has fewer lines (%d) than there are sequences (%d)" % (state.shape[0], n))
    if state.shape[0] > _MOST:
        _fits(state.shape[0])
    dev = x.device
    _on(dev, state=state, x=x, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias,
        cache_indices=read, out_indices=write)
    y = _new(x)
    if n == 0:
        return y
    desc.B, desc.T, desc.N, desc.dt_softplus = n, 1, n, int(bool(dt_softplus))
    desc.state_lines = state.shape[0]
    st = _launch(dev, gdn_selective_state_update, desc, state, x, dt, A, B, C, D, z, dt_bias, read,
                 write, y)
    if st != 0:
        raise GdnError(st, "gdn_selective_state_update")
    return y


def gdn_causal_conv1d_bwd_workspace_size(desc: GdnConvDesc) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_causal_conv1d_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_causal_conv1d_bwd_workspace_size")
    return int(n)


def gdn_causal_conv1d_bwd(desc, x, weight, bias, initial, cu_seqlens, dy, dfinal, dx, dweight,
                          dbias, dinitial, workspace, workspace_bytes, stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_causal_conv1d_bwd(
        ctypes.byref(desc), *_addresses((x, weight, bias, initial, cu_seqlens, dy, dfinal, dx,
                                        dweight, dbias, dinitial, workspace)), workspace_bytes,
        _stream(stream)))


def causal_conv1d_bwd(x, weight, dy, bias=None, initial_state=None, dfinal_state=None,
                      cu_seqlens=None, activation=None, workspace=None):
    """Gradients of causal_conv1d's inputs on the current stream, given ``dy`` [B, T, C] and
    ``dfinal_state`` [N, W - 1, C] of the state lines afterwards (None: zero).  initial_state
    [N, W - 1, C]: the inputs before each sequence, its line before the forward (None: zeros).
    dx of tokens of a packed batch that no sequence has is not written.
    Returns (dx in x's dtype, dweight [C, W] and dbias [C] fp32, dinitial_state in x's dtype);
    dbias and dinitial_state are None where the input is None."""
    _validate_conv(x, weight, bias, None, None, None, cu_seqlens)
    _need(activation in ACTIVATIONS, ValueError, "activation must be None, 'none' or 'silu'")
    B, T, C = x.shape
    W = weight.shape[1]
    cu, N = _sequences(x, cu_seqlens)
    _fits(B, T, N, C)
    _need(dy is not None, TypeError, "dy is required")
    _like("dy", dy, x)
    lines = dict(initial_state=initial_state, dfinal_state=dfinal_state)
    for name, t in lines.items():
        if t is not None:
            _need(isinstance(t, torch.Tensor) and t.dtype == x.dtype, TypeError,
                  "%s must be a tensor of x's dtype %s" % (name, x.dtype))
            _need(tuple(t.shape) == (N, W - 1, C), ValueError,
                  "%s must be [N, W - 1, C] = %s" % (name, [N, W - 1, C]))
            lines[name] = t.contiguous()
    _on(x.device, x=x, dy=dy, workspace=workspace, **lines)
    weight, dy = weight.contiguous(), dy.contiguous()
    bias = None if bias is None else bias.contiguous()
    desc = GdnConvDesc(B=B, T=T, N=N, channels=C, width=W, dtype=_code(x),
                       activation=ACTIVATIONS[activation], state_lines=0)
    dev = x.device
    first = lines["initial_state"]
    dx, dweight, dbias, dinit = _new(x), _new(weight), _new(bias), _new(first)
    if B == 0:
        return dx, dweight.zero_(), _zero(dbias), dinit
    need = gdn_causal_conv1d_bwd_workspace_size(desc)
    ws = _workspace(desc, 0, workspace, dev)
    if need and (ws is None or ws.numel() < need):
        ws = torch.empty(need, device=dev, dtype=torch.uint8)
    st = _launch(dev, gdn_causal_conv1d_bwd, desc, x, weight, bias, first, cu, dy,
                 lines["dfinal_state"], dx, dweight, dbias, dinit, ws,
                 0 if ws is None else ws.numel())
    if st != 0:
        raise GdnError(st, "gdn_causal_conv1d_bwd")
    return dx, dweight, dbias, dinit


def gdn_group_norm_workspace_size(desc: GdnNormDesc, backward=False) -> int:
    st = ctypes.c_int(0)
    n = load().gdn_group_norm_workspace_size(ctypes.byref(desc), int(bool(backward)),
                                             ctypes.byref(st))
    if st.value != 0:
        raise GdnError(st.value, "gdn_group_norm_workspace_size")
    return int(n)


def gdn_group_norm_fwd(desc, x, weight, bias, gate, y, mean, rstd, stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_group_norm_fwd(
        ctypes.byref(desc), *_addresses((x, weight, bias, gate, y, mean, rstd)),
        _stream(stream)))


def gdn_group_norm_bwd(desc, x, weight, bias, gate, mean, rstd, dy, dx, dweight, dbias, dgate,
                       stream=None) -> int:
    """Raw call (tensors, integer device addresses or None); returns the status code."""
    return int(load().gdn_group_norm_bwd(
        ctypes.byref(desc), *_addresses((x, weight, bias, gate, mean, rstd, dy, dx, dweight,
                                        dbias, dgate)), _stream(stream)))


def _norm_operands(x, num_groups, weight, bias, eps, activation, gate):
    if not isinstance(x, Tensor):
        raise TypeError("x must be a torch tensor")
    code, shape = _CODES.get(x.dtype), x.shape
    if code is None:
        raise TypeError("x must be bf16 or fp32, got %s" % x.dtype)
    if len(shape) < 2 or shape[-1] == 0:
        raise ValueError("x must be [samples, channels] or [samples, ..., channels]")
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be None, 'none' or 'silu'")
    C = shape[-1]
    if not isinstance(num_groups, int) or num_groups <= 0 or C % num_groups:
        raise ValueError("num_groups must divide the %d channels, got %r" % (C, num_groups))
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    positions = 1
    for n in shape[1:-1]:
        positions *= n
    if not 0 < x.numel() <= _MOST:  # else no axis is longer either
        _fits(shape[0], positions, C)
    weight, bias = _f32("weight", weight, (C,)), _f32("bias", bias, (C,))
    _like("gate", gate, x)
    if gate is not None:
        gate = gate.contiguous()
    desc = GdnNormDesc(shape[0], positions, C, num_groups, code, ACTIVATIONS[activation], eps, None,
                       0)
    return desc, x.contiguous(), weight, bias, gate


def group_norm(x, num_groups, weight=None, bias=None, eps=1e-5, activation=None, gate=None,
               workspace=None):
    """Channels-last group norm with an activation or a gate on the current stream.

    x: [samples, channels] (a token's heads: every row by itself) or [samples, ..., channels]
    (statistics over a sample's positions and a group's channels), bf16 or fp32; weight, bias
    [channels] fp32 or None; gate: x's shape and dtype, or None.  y = act(u) without a gate and
    u act(gate) with one, u the normalised, scaled and shifted x.  Returns (y, mean, rstd), mean
    and rstd [samples, num_groups] fp32 (NaN where there are no positions)."""
    desc, x, weight, bias, gate = _norm_operands(x, num_groups, weight, bias, eps, activation,
                                                 gate)
    dev = x.device
    _on(dev, x=x, weight=weight, bias=bias, gate=gate, workspace=workspace)
    y = _new(x)
    mean = x.new_empty((x.shape[0], num_groups), dtype=torch.float32)
    rstd = _new(mean)
    ws = _workspace(desc, gdn_group_norm_workspace_size(desc), workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_group_norm_fwd, desc, x, weight, bias, gate, y, mean, rstd)
    if st != 0:
        raise GdnError(st, "gdn_group_norm_fwd")
    return y, mean, rstd


def group_norm_bwd(dy, x, num_groups, mean, rstd, weight=None, bias=None, activation=None,
                   gate=None, workspace=None):
    """Gradients of group_norm's inputs on the current stream, from dy, the forward's inputs and
    its mean and rstd.  Returns (dx, dweight, dbias, dgate): dx and dgate in x's dtype, dweight
    and dbias [channels] fp32; None where the input is None."""
    desc, x, weight, bias, gate = _norm_operands(x, num_groups, weight, bias, 0.0, activation,
                                                 gate)
    _need(dy is not None, TypeError, "dy is required")
    _like("dy", dy, x)
    _need(mean is not None and rstd is not None, TypeError, "mean and rstd are required")
    mean = _f32("mean", mean, (x.shape[0], num_groups))
    rstd = _f32("rstd", rstd, (x.shape[0], num_groups))
    dev = x.device
    _on(dev, x=x, dy=dy, mean=mean, rstd=rstd, weight=weight, bias=bias, gate=gate,
        workspace=workspace)
    dy = dy.contiguous()
    dx, dweight, dbias, dgate = map(_new, (x, weight, bias, gate))
    ws = _workspace(desc, gdn_group_norm_workspace_size(desc, True), workspace, dev)  # noqa: F841
    st = _launch(dev, gdn_group_norm_bwd, desc, x, weight, bias, gate, mean, rstd, dy, dx, dweight,
                 dbias, dgate)
    if st != 0:
        raise GdnError(st, "gdn_group_norm_bwd")
    return dx, dweight, dbias, dgate
