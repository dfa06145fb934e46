"""The oracles of the convolution's gradient and of the group norm (no GPU): against the forward
oracle's differences and against identities."""
import numpy as np
import pytest

from oracle import conv1d, norm
from oracle.conv1d_backward import causal_conv1d_backward


def differences(f, v, e=1e-5):
    out = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = v[i]
        v[i] = keep + e
        hi = f()
        v[i] = keep - e
        lo = f()
        v[i] = keep
        out[i] = (hi - lo) / (2 * e)
    return out


@pytest.mark.parametrize("lens,W,silu", [(None, 4, True), ([3, 0, 1, 2], 3, True), ([1, 5], 2, False)])
def test_convolution_gradient_against_differences(lens, W, silu):
    r = np.random.default_rng(3)
    B, T, C = (2, 5, 3) if lens is None else (1, sum(lens), 3)
    N = B if lens is None else len(lens)
    cu = None if lens is None else np.cumsum([0] + lens)
    x, w, b = r.standard_normal((B, T, C)), r.standard_normal((C, W)), r.standard_normal(C)
    first = r.standard_normal((N, W - 1, C))
    dy, dfinal = r.standard_normal(x.shape), r.standard_normal(first.shape)

    def loss():
        y, last = conv1d.causal_conv1d(x, w, b, first, None, None, cu, "silu" if silu else "none")
        return (y * dy).sum() + (last * dfinal).sum()

    dx, dw, db, dfirst = causal_conv1d_backward(x, w, dy, b, first, dfinal, cu, silu)
    for got, v in ((dx, x), (dw, w), (db, b), (dfirst, first)):
        assert np.allclose(got, differences(loss, v), rtol=1e-6, atol=1e-8)


def test_norm_identities():
    r = np.random.default_rng(4)
    x = r.standard_normal((3, 5, 12)) * 2 + 7
    y, mean, rstd = norm.group_norm(x, 4, eps=0.0)
    g = y.reshape(3, 5, 4, 3)
    assert np.allclose(g.mean((1, 3)), 0, atol=1e-12) and np.allclose((g ** 2).mean((1, 3)), 1)
    y2, _, _ = norm.group_norm(3 * x - 5, 4, eps=0.0)  # blind to scale and shift
    assert np.allclose(y, y2)


@pytest.mark.parametrize("silu,gated", [(False, False), (True, False), (True, True), (False, True)])
def test_norm_gradient_against_differences(silu, gated):
    r = np.random.default_rng(5)
    x, w, b = r.standard_normal((2, 3, 6)), r.standard_normal(6), r.standard_normal(6)
    gate = r.standard_normal(x.shape) if gated else None
    dy = r.standard_normal(x.shape)

    def loss():
        return (norm.group_norm(x, 2, w, b, 1e-3, silu, gate)[0] * dy).sum()

    dx, dw, db, dgate = norm.group_norm_backward(dy, x, 2, w, b, 1e-3, silu, gate)
    for got, v in ((dx, x), (dw, w), (db, b)) + (((dgate, gate),) if gated else ()):
        assert np.allclose(got, differences(loss, v), rtol=1e-6, atol=1e-8)
