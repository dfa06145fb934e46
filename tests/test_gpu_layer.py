"""GPU parity of the convolution's gradient and of the group norm against the fp64 oracles.

Tolerances, relative L2 over each tensor.  A value here is a short chain of fp32 operations (at
most 4 taps, an activation, the statistics), each within 2^-23 of it: about 20 of them, 2.4e-6,
with cancellation of up to 4 between the terms of a gradient: 1e-5 in fp32.  Sums over tokens are
joined from partial sums, which adds no more than the terms' own error.  bf16 outputs: one rounding
to 8 significant bits more, 2^-8 + 1e-5.
"""
import numpy as np
import pytest
import torch

from oracle import norm
from oracle.conv1d_backward import causal_conv1d_backward

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL_F32 = 1e-5
TOL = {"f32": TOL_F32, "bf16": 2.0 ** -8 + 1e-5}


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def check(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    if got.size:
        d = np.linalg.norm(ref)
        e = float(np.linalg.norm(got - ref) / (d if d else 1.0))
        assert e <= tol, "%s: relative L2 %.3g over %.3g" % (name, e, tol)


# --- the convolution's gradient ---------------------------------------------------------------

CONV = [
    # B, T, C, W, dtype, silu, bias, initial, lens
    (1, 1, 8, 4, "f32", True, True, True, None),
    (3, 70, 2112, 4, "bf16", True, True, True, None),
    (2, 33, 2112, 3, "f32", False, True, False, None),
    (2, 65, 64, 2, "bf16", True, False, False, None),
    (4, 2, 2048, 4, "bf16", False, True, True, None),
    (2, 600, 24, 4, "f32", True, True, True, None),       # several token blocks
    (1, 0, 40, 4, "f32", True, True, True, [5, 0, 1, 64, 2, 3, 0, 300]),
    (1, 0, 40, 3, "bf16", True, True, False, [1, 1, 2, 1, 0, 9]),
    (1, 0, 16, 2, "f32", False, False, True, [0, 0, 17]),
    (1, 0, 8, 4, "f32", True, True, True, [0, 0]),
]


@pytest.mark.parametrize("B,T,C,W,dtype,silu,bias,initial,lens", CONV)
def test_conv_gradient_matches_oracle(B, T, C, W, dtype, silu, bias, initial, lens):
    import gated_deltanet_chunked_02_amd as gdn
    g = torch.Generator().manual_seed(C + W + T)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DTYPES[dtype]
    if lens is not None:
        T = sum(lens)
    N = B if lens is None else len(lens)
    x, dy = n(B, T, C).to(dt), n(B, T, C).to(dt)
    w, b = n(C, W) * W ** -0.5, n(C) * 0.1 if bias else None
    first = n(N, W - 1, C).to(dt) if initial else None
    dfinal = n(N, W - 1, C).to(dt) if initial else None
    cu = None if lens is None else torch.tensor(np.cumsum([0] + lens), dtype=torch.int32)
    mv = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = gdn.causal_conv1d_bwd(mv(x), mv(w), mv(dy), bias=mv(b), initial_state=mv(first),
                                dfinal_state=mv(dfinal), cu_seqlens=mv(cu),
                                activation="silu" if silu else None)
    torch.cuda.synchronize()
    ref = causal_conv1d_backward(host(x), host(w), host(dy), host(b), host(first), host(dfinal),
                                 None if cu is None else cu.numpy(), silu)
    check("dx", got[0], ref[0], TOL[dtype])
    check("dweight", got[1], ref[1], TOL_F32)
    if bias:
        check("dbias", got[2], ref[2], TOL_F32)
    else:
        assert got[2] is None
    if initial:
        check("dinitial", got[3], ref[3], TOL[dtype])
    else:
        assert got[3] is None


def test_conv_gradient_same_bits_on_another_stream():
    import gated_deltanet_chunked_02_amd as gdn
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 500, 256, generator=g, device="cuda")
    dy = torch.randn(2, 500, 256, generator=g, device="cuda")
    w = torch.randn(256, 4, generator=g, device="cuda")
    a = gdn.causal_conv1d_bwd(x, w, dy, activation="silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = gdn.causal_conv1d_bwd(x, w, dy, activation="silu")
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --- the group norm ---------------------------------------------------------------------------

NORM = [
    # shape, groups, dtype, silu, gated, affine
    ((1, 1), 1, "f32", False, False, True),
    ((5, 64), 1, "bf16", True, False, True),
    ((70, 4096), 32, "bf16", True, True, True),
    ((33, 320), 32, "f32", True, False, True),        # 10 channels a group: short vectors
    ((9, 37 * 3), 3, "bf16", True, True, True),       # odd: single values
    ((7, 96), 96, "f32", True, False, True),          # a channel a group: xhat is zero
    ((3, 8192), 1, "bf16", False, False, False),
    ((2, 12288), 1, "f32", True, True, True),         # a row over the whole workgroup's registers
    ((2, 5000), 1, "bf16", True, False, True),
    ((3, 1003), 1, "bf16", True, True, True),
    ((300, 24), 3, "f32", False, True, True),
    ((2, 63, 320), 32, "f32", True, False, True),
    ((2, 7, 9, 320), 32, "bf16", True, True, True),
    ((1, 1000, 64), 4, "bf16", True, False, True),    # several pieces of the positions
    ((3, 500, 37), 1, "f32", True, False, False),
    ((2, 4096, 40), 5, "f32", False, False, True),
    ((1, 300, 4096), 32, "bf16", True, False, True),  # several workgroups a row
    ((4, 2, 16), 2, "f32", True, True, True),
]


def norm_inputs(shape, groups, dtype, gated, affine, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DTYPES[dtype]
    C = shape[-1]
    return dict(x=(n(*shape) * torch.exp(0.5 * n(C)) + 0.3).to(dt), dy=n(*shape).to(dt),
                weight=1 + 0.1 * n(C) if affine else None, bias=0.1 * n(C) if affine else None,
                gate=n(*shape).to(dt) if gated else None)


@pytest.mark.parametrize("shape,groups,dtype,silu,gated,affine", NORM)
def test_norm_matches_oracle(shape, groups, dtype, silu, gated, affine):
    import gated_deltanet_chunked_02_amd as gdn
    p = norm_inputs(shape, groups, dtype, gated, affine)
    q = {k: None if v is None else v.cuda() for k, v in p.items()}
    act = "silu" if silu else None
    y, mean, rstd = gdn.group_norm(q["x"], groups, q["weight"], q["bias"], 1e-5, act, q["gate"])
    grads = gdn.group_norm_bwd(q["dy"], q["x"], groups, mean, rstd, q["weight"], q["bias"], act,
                               q["gate"])
    torch.cuda.synchronize()
    args = (host(p["x"]), groups, host(p["weight"]), host(p["bias"]), 1e-5, silu, host(p["gate"]))
    y_ref, mean_ref, rstd_ref = norm.group_norm(*args)
    check("y", y, y_ref, TOL[dtype])
    check("mean", mean, mean_ref, TOL_F32)
    check("rstd", rstd, rstd_ref, TOL_F32)
    ref = norm.group_norm_backward(host(p["dy"]), *args)
    if shape[-1] == groups and len(shape) == 2:
        # one value a group: dx is rstd (dhat - dhat - 0), zero but for rounding of dhat
        assert float(grads[0].abs().max()) <= 1e-6 * float(rstd.max())
    else:
        check("dx", grads[0], ref[0], TOL[dtype])
    for k, i in (("weight", 1), ("bias", 2)):
        if p[k] is None:
            assert grads[i] is None
        else:
            check("d" + k, grads[i], ref[i], TOL_F32)
    if gated:
        check("dgate", grads[3], ref[3], TOL[dtype])
    else:
        assert grads[3] is None


@pytest.mark.parametrize("shape,groups", [((40, 256), 8), ((2, 900, 64), 8), ((2, 20, 64), 8)])
def test_norm_far_from_zero(shape, groups):
    """A mean of 4096 times the deviation: the variance must come from differences, not from large
    sums.  The inputs carry the mean exactly, so x - mean loses no more than 4096 x 2^-23 x 2 of
    the deviation: 1e-3."""
    import gated_deltanet_chunked_02_amd as gdn
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(2)) + 4096.0
    y, mean, rstd = gdn.group_norm(x.cuda(), groups)
    y_ref, _, rstd_ref = norm.group_norm(host(x), groups)
    check("y", y, y_ref, 1e-3)
    check("rstd", rstd, rstd_ref, 1e-3)


@pytest.mark.parametrize("shape", [(3, 64), (2, 600, 64), (2, 5, 64)])
def test_norm_of_constants_and_of_one_infinity(shape):
    import gated_deltanet_chunked_02_amd as gdn
    x = torch.full(shape, 3.0).cuda()
    y, mean, rstd = gdn.group_norm(x, 4, eps=1e-5)
    assert not y.any() and torch.all(mean == 3.0)
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)).cuda()
    clean = gdn.group_norm(x, 4)[0]
    x[(0,) * (len(shape) - 1) + (17,)] = float("inf")  # sample 0, group 1
    y = gdn.group_norm(x, 4)[0]
    assert torch.isnan(y[0, ..., 16:32]).any()
    y[0, ..., 16:32], clean[0, ..., 16:32] = 0, 0
    assert torch.equal(y, clean)  # other groups and samples untouched


def test_norm_on_unaligned_rows_and_another_stream():
    import gated_deltanet_chunked_02_amd as gdn
    for shape, groups in (((50, 256), 8), ((2, 700, 64), 4)):
        p = norm_inputs(shape, groups, "bf16", True, True, seed=3)
        q = {k: v.cuda() for k, v in p.items()}
        args = lambda x: (x, groups, q["weight"], q["bias"], 1e-5, "silu", q["gate"])  # noqa: E731
        y, mean, rstd = gdn.group_norm(*args(q["x"]))
        n = q["x"].numel()
        off = torch.zeros(n + 1, dtype=torch.bfloat16, device="cuda")[1:].view(shape)
        off.copy_(q["x"])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            y2, mean2, rstd2 = gdn.group_norm(*args(off))
            g2 = gdn.group_norm_bwd(q["dy"], off, groups, mean2, rstd2, q["weight"], q["bias"],
                                    "silu", q["gate"])
        s.synchronize()
        check("y", y2, host(y), 2.0 ** -7)  # two roundings to bf16 of values 1e-5 apart
        check("mean", mean2, host(mean), TOL_F32)
        ref = norm.group_norm_backward(host(p["dy"]), host(p["x"]), groups, host(p["weight"]),
                                       host(p["bias"]), 1e-5, True, host(p["gate"]))
        check("dx", g2[0], ref[0], TOL["bf16"])
        check("dweight", g2[1], ref[1], TOL_F32)
        check("dgate", g2[3], ref[3], TOL["bf16"])


def test_norm_of_nothing():
    import gated_deltanet_chunked_02_amd as gdn
    x = torch.zeros(0, 64, device="cuda")
    y, mean, rstd = gdn.group_norm(x, 4)
    w = torch.ones(64, device="cuda")
    dx, dw, _, _ = gdn.group_norm_bwd(x, x, 4, mean, rstd, weight=w)
    torch.cuda.synchronize()
    assert y.shape == dx.shape == (0, 64) and not dw.any()
