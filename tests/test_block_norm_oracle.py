"""Pins of the block norm oracle: closed forms and differences."""
import numpy as np
import pytest

from oracle import block_norm as bn


def make(seed=0, R=4, C=7):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    return dict(x=n((R, C)), h=n((R, C)), weight=n(C), post_norm=True, post=n(C), gate=n((R, C)),
                silu=True, scale=n(C), residual_scale=0.6, eps=1e-3), n((R, C)), n((R, C))


def test_closed_forms():
    p, _, _ = make()
    out, y, rstd1, rstd2 = bn.block_norm(p["x"], eps=0.0)
    assert np.array_equal(out, p["x"]) and np.allclose((y ** 2).mean(-1), 1.0)
    assert np.allclose(rstd2, (p["x"] ** 2).mean(-1) ** -0.5)
    # without a norm, a gate of ones and a stream of zeros, the addition is the block's output
    out, _, rstd1, _ = bn.block_norm(0 * p["x"], p["h"], gate=np.ones((4, 7)), residual_scale=2.0)
    assert np.allclose(out, 2 * p["h"]) and np.all(rstd1 == 1.0)
    # a post-norm forgets its input's size
    a = bn.block_norm(**dict(p, eps=0.0))
    b = bn.block_norm(**dict(p, eps=0.0, h=3 * p["h"]))
    assert np.allclose(a[0], b[0]) and np.allclose(a[2], 3 * b[2])
    # silu: g - silu(g) = -silu(-g) ... the two halves of a gate
    zero = dict(p, x=0 * p["x"])
    up = bn.block_norm(**zero)[0]
    down = bn.block_norm(**dict(zero, gate=-p["gate"]))[0]
    plain = bn.block_norm(**dict(zero, silu=False))[0]
    assert np.allclose(up - down, plain)


@pytest.mark.parametrize("change", [{}, dict(post_norm=False, post=None), dict(gate=None),
                                    dict(silu=False), dict(scale=None, weight=None)])
def test_gradients_equal_differences(change):
    p, dy, dx = make(seed=2)
    p.update(change)

    def loss(**c):
        out, y, _, _ = bn.block_norm(**dict(p, **c))
        return (out * dx).sum() + (y * dy).sum()

    args = {k: v for k, v in p.items()}
    got = bn.block_norm_backward(dy, dx, **args)
    r = np.random.default_rng(1)
    for name in ("x", "h", "gate", "weight", "post", "scale"):
        if p[name] is None:
            continue
        d, eps = r.standard_normal(p[name].shape), 1e-6
        want = (loss(**{name: p[name] + eps * d}) - loss(**{name: p[name] - eps * d})) / (2 * eps)
        assert abs(want - (got["d" + name] * d).sum()) <= 1e-6 * max(1.0, abs(want)), name
