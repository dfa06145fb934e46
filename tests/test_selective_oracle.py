"""The selective scan's oracle (no GPU): against a closed form, against a dense sum, and its
gradients against differences."""
import numpy as np
import pytest

from oracle import selective


def make(B=1, T=5, C=6, G=2, S=3, seed=0, lens=None):
    r = np.random.default_rng(seed)
    p = dict(x=r.standard_normal((B, T, C)), dt=r.standard_normal((B, T, C)) * 0.5 - 1.0,
             A=-np.exp(r.standard_normal((C, S)) * 0.3), B=r.standard_normal((B, T, G, S)),
             C=r.standard_normal((B, T, G, S)), D=r.standard_normal(C),
             z=r.standard_normal((B, T, C)), dt_bias=r.standard_normal(C) * 0.1)
    n = B if lens is None else len(lens)
    p["h0"] = r.standard_normal((n, C, S))
    p["cu"] = None if lens is None else np.cumsum([0] + lens)
    return p


def test_constant_inputs_follow_the_geometric_series():
    T, a = 7, np.exp(-0.5 * 2.0)
    y, ht = selective.scan(np.ones((1, T, 1)), np.full((1, T, 1), 0.5), np.array([[-2.0]]),
                           np.ones((1, T, 1, 1)), np.ones((1, T, 1, 1)))
    want = 0.5 * (1 - a ** np.arange(1, T + 1)) / (1 - a)
    assert np.allclose(y[0, :, 0], want, rtol=1e-13)
    assert np.allclose(ht[0, 0, 0], want[-1], rtol=1e-13)


def test_equals_the_sum_over_earlier_tokens():
    p = make(T=9, seed=3)
    y, ht = selective.scan(dt_softplus=True, **p)
    step = np.logaddexp(0, p["dt"] + p["dt_bias"])[0]
    per = p["A"].shape[0] // p["B"].shape[2]
    for c in range(6):
        cum = np.concatenate([[0.0], np.cumsum(step[:, c])])
        for t in range(9):
            h = np.exp(cum[t + 1] * p["A"][c]) * p["h0"][0, c]
            for j in range(t + 1):
                h = h + np.exp((cum[t + 1] - cum[j + 1]) * p["A"][c]) * step[j, c] * \
                    p["x"][0, j, c] * p["B"][0, j, c // per]
            want = (h @ p["C"][0, t, c // per] + p["D"][c] * p["x"][0, t, c])
            z = p["z"][0, t, c]
            assert np.isclose(y[0, t, c], want * z / (1 + np.exp(-z)), rtol=1e-11)
        assert np.allclose(ht[0, c], h, rtol=1e-11)


def test_packed_is_each_sequence_alone_and_an_empty_one_keeps_its_state():
    lens = [3, 0, 1, 5]
    p = make(T=9, seed=4, lens=lens)
    y, ht = selective.scan(dt_softplus=True, **p)
    for n, (a, e) in enumerate(zip(p["cu"][:-1], p["cu"][1:])):
        cut = {k: p[k][:, a:e] for k in ("x", "dt", "B", "C", "z")}
        y1, h1 = selective.scan(A=p["A"], D=p["D"], dt_bias=p["dt_bias"], dt_softplus=True,
                                h0=p["h0"][n:n + 1], **cut)
        assert np.array_equal(y[:, a:e], y1) and np.array_equal(ht[n], h1[0])
    assert np.array_equal(ht[1], p["h0"][1])


@pytest.mark.parametrize("lens", [None, [2, 0, 3]])
def test_gradients_against_differences(lens):
    p = make(T=5, C=4, G=2, S=2, seed=7, lens=lens)
    r = np.random.default_rng(8)
    dy, dht = r.standard_normal(p["x"].shape), r.standard_normal(p["h0"].shape)

    def loss(q):
        y, ht = selective.scan(dt_softplus=True, **q)
        return (y * dy).sum() + (ht * dht).sum()

    args = {k: p[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0", "cu")}
    g = selective.scan_backward(dy=dy, dht=dht, dt_softplus=True, **args)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="dbias",
                 h0="dh0")
    for k, gk in names.items():
        num = np.zeros_like(p[k])
        it = np.nditer(p[k], flags=["multi_index"])
        for _ in it:
            i = it.multi_index
            vals = []
            for s in (1e-5, -1e-5):
                q = {**p, k: p[k].copy()}
                q[k][i] += s
                vals.append(loss(q))
            num[i] = (vals[0] - vals[1]) / 2e-5
        assert np.allclose(g[gk], num, rtol=1e-6, atol=1e-8), k
