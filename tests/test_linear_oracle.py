"""Pins of the linear attention oracle: closed forms, the quadratic form, differences."""
import numpy as np
import pytest

from oracle import linear


def make(B=2, T=9, H=4, Hg=2, Dk=3, Dv=5, head=False, seed=0, cu=None):
    r = np.random.default_rng(seed)
    N = B if cu is None else len(cu) - 1
    g = -r.random(H) if head else -r.random((B, T, H))
    return dict(q=r.standard_normal((B, T, Hg, Dk)), k=r.standard_normal((B, T, Hg, Dk)),
                v=r.standard_normal((B, T, H, Dv)), g=g, scale=0.7,
                h0=r.standard_normal((N, H, Dk, Dv))), \
        r.standard_normal((B, T, H, Dv)), r.standard_normal((N, H, Dk, Dv))


def test_no_decay_is_a_causal_product():
    p, _, _ = make()
    p["g"] = np.zeros_like(p["g"])
    o, ht = linear.attention(**p)
    q, k = (np.repeat(p[x], 2, 2) for x in ("q", "k"))
    w = np.einsum("bihd,bjhd->bhij", q, k) * np.tril(np.ones((9, 9)))
    want = np.einsum("bhij,bjhd->bihd", w, p["v"]) + np.einsum("bihk,bhkd->bihd", q, p["h0"])
    assert np.allclose(o, 0.7 * want, atol=1e-12)
    assert np.allclose(ht, p["h0"] + np.einsum("bjhk,bjhd->bhkd", k, p["v"]), atol=1e-12)


def test_forgotten_states_leave_one_token():
    p, _, _ = make(head=True)
    p["g"] = np.full(4, -np.inf)
    o, ht = linear.attention(**p)
    q, k = (np.repeat(p[x], 2, 2) for x in ("q", "k"))
    assert np.allclose(o, 0.7 * (q * k).sum(-1, keepdims=True) * p["v"], atol=1e-12)
    assert np.allclose(ht, k[:, -1, :, :, None] * p["v"][:, -1, :, None, :], atol=1e-12)


def test_a_heads_decay_is_every_tokens():
    p, do, dht = make(head=True)
    q = dict(p, g=np.broadcast_to(p["g"], (2, 9, 4)))
    for a, b in zip(linear.attention(**p), linear.attention(**q)):
        assert np.array_equal(a, b)
    a = linear.attention_backward(**p, do=do, dht=dht)
    b = linear.attention_backward(**q, do=do, dht=dht)
    assert np.allclose(a["dg"], b["dg"].sum((0, 1)), atol=1e-12)


def test_packed_equals_sequences_apart_and_state_carries():
    cu = np.array([0, 4, 4, 9])
    p, _, _ = make(B=1, cu=cu)
    o, ht = linear.attention(**p, cu=cu)
    for n, (a, e) in enumerate(zip(cu, cu[1:])):
        part = {x: p[x][:, a:e] for x in ("q", "k", "v", "g")}
        o1, h1 = linear.attention(**part, scale=0.7, h0=p["h0"][n:n + 1])
        assert np.allclose(o[:, a:e], o1, atol=1e-12) and np.allclose(ht[n], h1[0], atol=1e-12)
    p, _, _ = make()
    o, ht = linear.attention(**p)
    cut = lambda a, e: {x: p[x][:, a:e] for x in ("q", "k", "v", "g")}  # noqa: E731
    o1, h1 = linear.attention(**cut(0, 5), scale=0.7, h0=p["h0"])
    o2, h2 = linear.attention(**cut(5, 9), scale=0.7, h0=h1)
    assert np.allclose(o, np.concatenate([o1, o2], 1), atol=1e-12)
    assert np.allclose(ht, h2, atol=1e-12)


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 4, 4, 9]])
def test_gradients_equal_differences(head, cu):
    p, do, dht = make(B=2 if cu is None else 1, head=head, cu=cu, seed=3)

    def loss(**change):
        o, ht = linear.attention(**dict(p, **change), cu=cu)
        return (o * do).sum() + (ht * dht).sum()

    got = linear.attention_backward(**p, do=do, dht=dht, cu=cu)
    r = np.random.default_rng(1)
    for name in ("q", "k", "v", "g", "h0"):
        d = r.standard_normal(p[name].shape)
        eps = 1e-5
        want = (loss(**{name: p[name] + eps * d}) - loss(**{name: p[name] - eps * d})) / (2 * eps)
        have = (got["d" + name] * d).sum()
        assert abs(want - have) <= 1e-6 * max(1.0, abs(want)), name
    # an oracle without the initial state's share of dg is caught by the same check
    d = np.ones_like(p["g"])
    wrong = linear.attention_backward(**dict(p, h0=np.zeros_like(p["h0"])), do=do, dht=dht, cu=cu)
    want = (loss(g=p["g"] + 1e-5 * d) - loss(g=p["g"] - 1e-5 * d)) / 2e-5
    assert abs(want - (wrong["dg"] * d).sum()) > 1e-3
