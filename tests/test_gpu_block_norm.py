"""GPU parity of the block norm and its gradient against the fp64 oracle.

Tolerances, relative L2 over each tensor.  fp32: a row's sum of squares is 8 values a thread and a
tree of at most 10 more, 18 roundings of 2^-24, half of it after the root; an output adds about ten
operations, the exponential and reciprocal of the gate among them: 30 x 2^-24 = 2e-6, gradients go
through two norms and a sum over rows: 5e-6 forward, 1e-5 backward.  bf16: one rounding of each
output, at most 2^-8 of a value, more.
"""
import numpy as np
import pytest
import torch

from oracle import block_norm as bn

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def make(R, C, dtype="f32", residual=None, post=True, gate=True, silu=True, scale=True,
         weight=True, seed=0, shape=None):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    dt, rt = DTYPES[dtype], DTYPES[residual or dtype]
    shape = shape or (R, C)
    p = dict(x=(n(*shape) * 2).to(rt), h=n(*shape).to(dt), post_norm=post,
             post=1 + 0.1 * n(C) if post else None, gate=n(*shape).to(dt) if gate else None,
             silu=silu, scale=0.3 + 0.1 * n(C) if scale else None,
             weight=1 + 0.1 * n(C) if weight else None, residual_scale=0.7)
    return p, n(*shape).to(dt), n(*shape).to(rt)


def kwargs(p, move=lambda t: t):
    return dict(weight=move(p["weight"]), post_norm=p["post_norm"], post_weight=move(p["post"]),
                gate=move(p["gate"]), activation="silu" if p["silu"] else None,
                scale=move(p["scale"]), residual_scale=p["residual_scale"])


def oracle_args(p):
    return {k: host(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def cuda(t):
    return None if t is None else t.cuda()


def check(name, got, ref, tol, size=0.0):
    got = host(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    norm = max(np.linalg.norm(ref), size)
    e = np.linalg.norm(got - ref) / (norm if norm else 1.0)
    assert e <= tol, "%s: relative L2 %.3g over %.3g" % (name, e, tol)


def tol(t, base):
    return base + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0)


def first_terms(p, dy, ref, dR):
    """The norms of rstd du in dx and in dh."""
    one = lambda t: 1.0 if t is None else host(t)  # noqa: E731
    g = one(p["gate"])
    act = g / (1.0 + np.exp(-g)) if p["silu"] and p["gate"] is not None else g
    dh = ref[2][..., None] * dR * p["residual_scale"] * one(p["scale"]) * act * one(p["post"])
    return dict(dx=np.linalg.norm(ref[3][..., None] * host(dy) * one(p["weight"])),
                dh=np.linalg.norm(dh))


def check_both(p, dy, dx, eps=1e-5):
    import gated_deltanet_chunked_02_amd as gdn
    x, h, kw = cuda(p["x"]), cuda(p["h"]), kwargs(p, cuda)
    out, y, r1, r2 = gdn.block_norm(x, h, eps=eps, **kw)
    grads = gdn.block_norm_bwd(cuda(dy), cuda(dx), x, h, r1, r2, **kw)
    torch.cuda.synchronize()
    ref = bn.block_norm(**oracle_args(p), eps=eps)
    check("x", out, ref[0], tol(out, 5e-6))
    check("y", y, ref[1], tol(y, 5e-6))
    if p["post_norm"]:
        check("post_rstd", r1, ref[2], 5e-6)
    check("rstd", r2, ref[3], 5e-6)
    want = bn.block_norm_backward(host(dy), host(dx), **oracle_args(p), eps=eps)
    given = dict(dx="x", dh="h", dgate="gate", dweight="weight", dpost="post", dscale="scale")
    size = first_terms(p, dy, ref, want["dx"])
    for (name, of), got in zip(given.items(), grads):
        if p[of] is None:
            assert got is None, name
        else:
            check(name, got, want[name], tol(got, 1e-5), size.get(name, 0.0))


@pytest.mark.parametrize("dtype,residual", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 8), (3, 2), (5, 7), (37, 64), (130, 100), (9, 511),
                                 (4, 512), (6, 513), (33, 1000), (7, 770), (5, 2048), (3, 4095),
                                 (3, 4104), (2, 8192), (3, 8193), (2, 20000)])
def test_matches_oracle(R, C, dtype, residual):
    check_both(*make(R, C, dtype, residual, seed=R + C))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [72, 1030, 9000])
@pytest.mark.parametrize("post,gate,silu,scale,weight", [
    (False, False, False, False, False), (True, False, False, False, True),
    (False, True, True, True, False), (True, True, False, False, True),
    (False, True, False, True, True), (True, False, False, True, False)])
def test_every_part_is_optional(C, post, gate, silu, scale, weight, dtype):
    p, dy, dx = make(11, C, dtype, None, post, gate, silu, scale, weight, seed=C)
    check_both(p, dy, dx)


def test_many_rows():
    """More rows than workgroups, of one wave and of several."""
    for R, C in ((20000, 40), (5000, 600)):
        check_both(*make(R, C, "bf16", "f32", seed=R))


@pytest.mark.parametrize("C", [96, 1031, 9000])
def test_first_and_last_norms(C):
    """No block's output yet (the first pre-norm), and none after (no y)."""
    import gated_deltanet_chunked_02_amd as gdn
    p, dy, dx = make(13, C, "bf16", "f32", seed=C)
    x, w = p["x"].cuda(), p["weight"].cuda()
    out, y, r1, r2 = gdn.block_norm(x, weight=w, dtype=torch.bfloat16)
    assert out is x and r1 is None and y.dtype == torch.bfloat16
    ref = bn.block_norm(host(p["x"]), weight=host(p["weight"]))
    check("y", y, ref[1], 2.0 ** -8 + 5e-6)
    for d in (dx, None):
        grads = gdn.block_norm_bwd(dy.cuda(), cuda(d), x, None, None, r2, weight=w)
        want = bn.block_norm_backward(host(dy), host(d), host(p["x"]), weight=host(p["weight"]))
        check("dx", grads[0], want["dx"], 1e-5)
        check("dweight", grads[3], want["dweight"], 1e-5)
        assert grads[1] is None and grads[2] is None and grads[4] is None and grads[5] is None
    p["weight"] = None
    kw = kwargs(p, cuda)
    out, y, r1, r2 = gdn.block_norm(x, p["h"].cuda(), pre_norm=False, **kw)
    assert y is None and r2 is None
    check("x", out, bn.block_norm(**oracle_args(p))[0], 5e-6)
    grads = gdn.block_norm_bwd(None, dx.cuda(), x, p["h"].cuda(), r1, None, **kw)
    want = bn.block_norm_backward(None, host(dx), **oracle_args(p))
    for name, got in zip(("dx", "dh", "dgate", None, "dpost", "dscale"), grads):
        if name:
            check(name, got, want[name], tol(got, 1e-5))


@pytest.mark.parametrize("C", [64, 1024, 9000])
def test_in_place_leading_axes_and_slices(C):
    import gated_deltanet_chunked_02_amd as gdn
    p, dy, dx = make(0, C, "bf16", "bf16", seed=3, shape=(2, 3, 5, C))
    kw = kwargs(p, cuda)
    x, h = p["x"].cuda(), p["h"].cuda()
    a = gdn.block_norm(x, h, **kw)
    assert a[0].shape == x.shape and a[3].shape == (2, 3, 5)
    # h and the gate as slices of one projection, at an odd element
    proj = torch.zeros(2, 3, 5, 2 * C + 1, dtype=torch.bfloat16, device="cuda")
    proj[..., 1:C + 1], proj[..., C + 1:] = h, kw["gate"]
    kw2 = dict(kw, gate=proj[..., C + 1:])
    b = gdn.block_norm(x, proj[..., 1:C + 1], **kw2)
    grads = gdn.block_norm_bwd(dy.cuda(), dx.cuda(), x, h, a[2], a[3], **kw)
    grads2 = gdn.block_norm_bwd(dy.cuda(), dx.cuda(), x, proj[..., 1:C + 1], a[2], a[3], **kw2)
    # where vectors do not fit, other threads hold the values: the 18 additions of a row's sum (see
    # above) come in another order, so the two agree to their roundings and not bit for bit
    for s, t in zip(a + tuple(grads), b + tuple(grads2)):
        check("strided", s, host(t), tol(s, 1e-5))
    # rows in another order are copied
    turned = h.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    c = gdn.block_norm(x, turned, **kw)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    again = x.clone()
    d = gdn.block_norm(again, h, inplace=True, **kw)
    assert d[0] is again and torch.equal(again, a[0]) and torch.equal(d[1], a[1])


def test_large_and_small_rows():
    """Values whose squares stay in fp32's range keep their accuracy; eps carries rows of zeros."""
    import gated_deltanet_chunked_02_amd as gdn
    p, dy, dx = make(6, 300, seed=1)
    p["x"] = p["x"] * torch.tensor([1e15, 1e-15, 1.0, 1e8, 1e-8, 0.0])[:, None]
    p["h"] = p["h"] * torch.tensor([1e15, 1e-15, 0.0, 1e-8, 1e8, 0.0])[:, None]
    out, y, _, _ = gdn.block_norm(p["x"].cuda(), p["h"].cuda(), eps=1e-12, **kwargs(p, cuda))
    ref = bn.block_norm(**oracle_args(p), eps=1e-12)
    for r in range(6):
        check("y", y[r], ref[1][r], 5e-6)
    assert not bool(y[5].any())


@pytest.mark.parametrize("C", [100, 1000, 9000])
def test_nan_stays_in_its_row(C):
    import gated_deltanet_chunked_02_amd as gdn
    p, dy, dx = make(12, C, "bf16", seed=4)
    kw = kwargs(p, cuda)
    x, h = p["x"].cuda(), p["h"].cuda()
    a = gdn.block_norm(x, h, **kw)
    ga = gdn.block_norm_bwd(dy.cuda(), dx.cuda(), x, h, a[2], a[3], **kw)
    h[3, 5], x[7, 2] = float("nan"), float("inf")
    b = gdn.block_norm(x, h, **kw)
    gb = gdn.block_norm_bwd(dy.cuda(), dx.cuda(), x, h, b[2], b[3], **kw)
    rest = [r for r in range(12) if r not in (3, 7)]
    for s, t in zip(a + tuple(ga[:3]), b + tuple(gb[:3])):
        assert torch.equal(s[rest], t[rest])
    assert bool(b[1][3].isnan().all()) and not bool(b[1][7].isfinite().all())


def test_no_rows():
    import gated_deltanet_chunked_02_amd as gdn
    p, dy, dx = make(0, 96, "bf16")
    kw = kwargs(p, cuda)
    out, y, r1, r2 = gdn.block_norm(p["x"].cuda(), p["h"].cuda(), **kw)
    assert out.shape == (0, 96) and y.shape == (0, 96) and r2.shape == (0,)
    grads = gdn.block_norm_bwd(dy.cuda(), dx.cuda(), p["x"].cuda(), p["h"].cuda(), r1, r2, **kw)
    for g in grads[3:]:
        assert g.shape == (96,) and not bool(g.any())


def test_reruns_streams_and_graphs_give_the_same_bits():
    import gated_deltanet_chunked_02_amd as gdn
    p, dy, dx = make(700, 1200, "bf16", "f32", seed=5)
    kw, x, h, dy, dx = kwargs(p, cuda), p["x"].cuda(), p["h"].cuda(), dy.cuda(), dx.cuda()

    def run():
        out, y, r1, r2 = gdn.block_norm(x, h, **kw)
        return [out, y, *gdn.block_norm_bwd(dy, dx, x, h, r1, r2, **kw)]

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_rows_past_2_to_31_elements():
    import gated_deltanet_chunked_02_amd as gdn
    R, C = 270000, 8192
    assert R * C > 2 ** 31
    r = torch.Generator(device="cuda").manual_seed(1)
    n = lambda: torch.randn(R, C, generator=r, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, h, dy = n(), n(), n()
    out, y, r1, r2 = gdn.block_norm(x, h, post_norm=True)
    dx, dh = gdn.block_norm_bwd(dy, None, x, h, r1, r2, post_norm=True)[:2]
    end = slice(R - 50, R)
    a = gdn.block_norm(x[end], h[end], post_norm=True)
    b = gdn.block_norm_bwd(dy[end], None, x[end], h[end], a[2], a[3], post_norm=True)
    for s, t in zip((out, y, r1, r2, dx, dh), (*a, *b[:2])):
        assert torch.equal(s[end], t)


@pytest.mark.parametrize("C", [64, 1024, 5120, 9000])
def test_parameters_at_any_address(C):
    """Parameters need their element's alignment only: slices of one buffer give the same bits."""
    import gated_deltanet_chunked_02_amd as gdn
    g = torch.Generator().manual_seed(C)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, h, gate, dy, dx = (n(37, C) for _ in range(5))
    w = [n(C) for _ in range(3)]
    buf = torch.zeros(3 * C + 9, device="cuda")
    odd = [buf[i * (C + 3) + 1:][:C] for i in range(3)]
    for a, b in zip(odd, w):
        a.copy_(b)
    got = []
    for weight, post, scale in (w, odd):
        kw = dict(weight=weight, post_norm=True, post_weight=post, gate=gate, activation="silu",
                  scale=scale)
        out, y, p, q = gdn.block_norm(x, h, **kw)
        got.append([out, y, p, q, *gdn.block_norm_bwd(dy, dx, x, h, p, q, **kw)])
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i
