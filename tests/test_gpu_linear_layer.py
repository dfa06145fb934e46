"""The example block, which runs linear attention and the block norm together as a model does."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_block_decodes_as_it_reads_and_runs():
    import linear_layer
    err, losses = linear_layer.main()
    # what the block adds goes through five tensors rounded to bf16 (y, its projection, o, the gated
    # norm, h), at slightly different values on the two sides, and the prompt's scores and the state
    # that meets q are rounded too: 7 x 2^-8
    assert err <= 7 * 2.0 ** -8, err
    assert all(math.isfinite(x) for x in losses)


def plain(layer, x, lens):
    """(x', the next block's input) by the formulas in x's precision, token by token."""
    rms = lambda t, w: t * (t.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w  # noqa: E731
    w = {n: getattr(layer, n) for n in layer.names}
    y = rms(x, w["pre"])
    q, k, v, gate, _, g = layer._project(y)
    rep = layer.heads // layer.shared
    q, k = (t.repeat_interleave(rep, 2) for t in (q, k))
    o = torch.zeros_like(v)
    for b in range(x.shape[0]):
        at = 0
        for n in lens or [x.shape[1]]:
            S, rows = x.new_zeros(layer.heads, layer.dk, layer.dv), []
            for t in range(at, at + n):
                S = S * g[b, t].exp()[:, None, None] + k[b, t, :, :, None] * v[b, t, :, None]
                rows.append(layer.dk ** -0.5 * (S * q[b, t, :, :, None]).sum(1))
            if rows:
                part = torch.zeros_like(v)
                part[b, at:at + n] = torch.stack(rows)
                o = o + part
            at += n
    mean = o.mean(-1, keepdim=True)
    n = (o - mean) * ((o - mean).square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    n = (n.flatten(2) * w["norm_w"] + w["norm_b"]) * torch.nn.functional.silu(gate)
    out = x + w["scale"] * rms(n @ w["w_out"], w["post"])
    return out, rms(out, w["following"])


class Double:
    """A layer's parameters in 64 bits on the host, as leaves, with its projection."""

    def __init__(self, layer):
        self.__dict__.update({n: getattr(layer, n) for n in ("heads", "shared", "dk", "dv", "names")})
        for n in layer.names:
            setattr(self, n, getattr(layer, n).double().cpu().requires_grad_())

    def _project(self, y):
        p = y @ self.w_in
        a, b = self.shared * self.dk, self.heads * self.dv
        q, k = (p[..., i * a:(i + 1) * a].unflatten(-1, (self.shared, self.dk)) for i in (0, 1))
        z = y @ self.w_g + 4.0
        return (q, k, p[..., 2 * a:2 * a + b].unflatten(-1, (self.heads, self.dv)),
                p[..., 2 * a + b:], z, torch.nn.functional.logsigmoid(z))


# fp32: twelve operations in a row (three norms, three products and the attention, there and back),
# each a sum of at most 320 terms: 12 x 320 x 2^-24 = 2.3e-4.  bf16: y, p, z, o, n, h there and dh, dn,
# do, dq (dk, dv), dz, dyin back are rounded, and within the attention two operands there and three
# back: 17 x 2^-8
TOLERANCE = {torch.float32: 12 * 320 * 2.0 ** -24, torch.bfloat16: 17 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,lens,heads,shared,dk,dv", [
    (37, None, 4, 2, 32, 24), (150, [1, 0, 70, 79], 2, 1, 64, 64), (3, None, 3, 3, 8, 40)])
def test_block_and_its_gradients(T, lens, heads, shared, dk, dv, dtype):
    import linear_layer
    B = 1 if lens else 2
    layer = linear_layer.LinearLayer(model=96, heads=heads, shared=shared, dk=dk, dv=dv, dtype=dtype,
                                     seed=T)
    r = torch.Generator().manual_seed(T + 1)
    x, dxo, dy = (torch.randn(B, T, 96, generator=r) for _ in range(3))
    dy = dy.to(dtype)
    cu = None
    if lens:
        cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    state = layer.pool(len(lens) if lens else B)
    got = layer.prompt(x.cuda(), state, cu_seqlens=cu)
    grads = layer.gradients(x.cuda(), dxo.cuda(), dy.cuda(), cu_seqlens=cu)

    ref = Double(layer)
    xd = x.double().requires_grad_()
    want = plain(ref, xd, lens)
    ((want[0] * dxo.double()).sum() + (want[1] * dy.double()).sum()).backward()
    leaves = [xd] + [getattr(ref, n) for n in ref.names]
    tol = TOLERANCE[dtype]
    for name, a, b in [("x_out", got[0], want[0]), ("y", got[1], want[1])] + [
            (n, a, b.grad) for n, a, b in zip(("x",) + layer.names, grads, leaves)]:
        a, b = a.double().cpu(), b.detach()
        assert a.shape == b.shape, name
        assert float((a - b).norm() / b.norm()) <= tol, name


@pytest.mark.parametrize("packed", [False, True])
def test_block_replays_from_a_graph(packed):
    """A prompt, a token and a gradient captured once and replayed on changed inputs give the eager
    calls' bits, the program's own work between the replays."""
    import linear_layer
    layer = linear_layer.LinearLayer(model=128, heads=4, shared=2, dk=64, dv=64, seed=2)
    r = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=r).cuda()  # noqa: E731
    B, T = (1, 900) if packed else (2, 450)
    cu = torch.tensor([0, 300, 301, 900], dtype=torch.int32, device="cuda") if packed else None
    seqs = 3 if packed else 2
    x, dxo, dy, one = n(B, T, 128), n(B, T, 128), n(B, T, 128).bfloat16(), n(seqs, 128)
    state, lines = layer.pool(seqs), torch.arange(seqs, dtype=torch.int32, device="cuda")

    def run():
        state.zero_()
        out, y = layer.prompt(x, state, cu_seqlens=cu)
        last, ylast = layer.token(one, state, lines)
        return [out, y, last, ylast, state, *layer.gradients(x, dxo, dy, cu_seqlens=cu)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(4):
        x.copy_(n(B, T, 128))
        one.copy_(n(seqs, 128))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for i, (a, b) in enumerate(zip(got, run())):
            assert torch.equal(a, b), i
