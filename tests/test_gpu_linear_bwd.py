"""GPU parity of linear attention's gradient against the fp64 oracle's.

Tolerances, relative L2 over each tensor.  fp32 results (dg and dh0 whatever the type): states and
their gradients each carry at most 5e-6 (see test_gpu_linear), a gradient is a product of both, 1e-5,
and dg adds four sums of a chunk's terms, each on a random walk of 64 roundings (8 x 2^-24): 2e-5.  bf16
outputs: one tensor rounded to bf16 on each path and then the output, 2 x 2^-8 + 2e-5; dv's state is
rounded on the way as well, but that is its path's one rounding.
"""
import pytest
import torch

from oracle import linear
from test_gpu_linear import DTYPES, LENS, check, dev, host, make, spans

pytestmark = pytest.mark.gpu

TOL_F32 = 2e-5
TOL = {"f32": TOL_F32, "bf16": 2 * 2.0 ** -8 + 2e-5}
NAMES = ("dq", "dk", "dv", "dg", "dh0")


def oracle_bwd(p, dht=True, scale=None):
    return linear.attention_backward(
        *(host(p[x]) for x in ("q", "k", "v", "g", "do")),
        scale=p["q"].shape[-1] ** -0.5 if scale is None else scale, h0=host(p["h0"]),
        dht=host(p["dht"]) if dht else None, cu=spans(p))


def run_bwd(p, dht=True, **kw):
    import gated_deltanet_chunked_02_amd as gdn
    q = dev(p)
    out = gdn.linear_attention_bwd(q["q"], q["k"], q["v"], q["g"], q["do"],
                                   dht=q["dht"] if dht else None, initial_state=q["h0"],
                                   cu_seqlens=q["cu"], **kw)
    torch.cuda.synchronize()
    return dict(zip(NAMES, out))


def check_all(p, got, ref, dtype):
    for x in NAMES:
        if x == "dh0" and p["h0"] is None:
            assert got[x] is None
        else:
            check(x, got[x], ref[x], TOL_F32 if x in ("dg", "dh0") else TOL[dtype])


BWD = [
    # B, T, H, Hg, Dk, Dv, head, h0, dht
    (1, 1, 1, 1, 8, 8, False, True, True),
    (1, 1, 2, 1, 64, 64, True, False, True),
    (2, 15, 3, 3, 64, 40, False, True, False),
    (2, 16, 4, 2, 16, 128, True, True, True),
    (1, 31, 2, 2, 96, 64, False, False, False),
    (1, 33, 2, 1, 128, 128, False, True, True),
    (3, 63, 5, 5, 40, 72, True, True, True),
    (1, 64, 2, 2, 64, 64, False, True, True),
    (1, 65, 6, 2, 128, 64, False, True, True),
    (2, 127, 4, 1, 64, 128, False, True, True),
    (1, 128, 2, 2, 128, 24, True, False, True),
    (1, 129, 2, 2, 72, 104, False, True, True),   # two segments, the second of one token
    (1, 700, 2, 1, 128, 128, False, True, True),
    (2, 300, 3, 3, 128, 96, True, True, True),
    (70, 3, 4, 4, 64, 64, False, True, True),     # more heads than run at once
    (5, 257, 64, 64, 32, 32, False, True, True),  # whole sequences of several chunks
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hg,Dk,Dv,head,h0,dht", BWD)
def test_gradients_match_oracle(B, T, H, Hg, Dk, Dv, head, h0, dht, dtype):
    p = make(B, T, H, Hg, Dk, Dv, dtype, head, h0, seed=B + T + Dk)
    check_all(p, run_bwd(p, dht=dht), oracle_bwd(p, dht=dht), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,head", [(2, False), (2, True), (96, False)])
def test_packed_gradients_match_oracle(lens, dtype, H, head):
    p = make(H=H, Hg=H // 2, Dk=16, Dv=32, dtype=dtype, head=head, lens=lens, seed=len(lens))
    got, ref = run_bwd(p), oracle_bwd(p)
    check_all(p, got, ref, dtype)
    for n, k in enumerate(lens):
        if k == 0:
            assert torch.equal(got["dh0"][n].cpu(), p["dht"][n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("worst", [-60.0, torch.finfo(torch.float32).min, -float("inf")])
def test_strong_decays(worst, dtype):
    p = make(2, 150, 3, 3, 64, 64, dtype, seed=4)
    r = torch.rand(p["g"].shape, generator=torch.Generator().manual_seed(5))
    p["g"] = torch.where(r < 0.1, torch.tensor(worst), p["g"])
    p["g"][0, 70:75] = worst
    got, ref = run_bwd(p), oracle_bwd(p)
    check_all(p, got, ref, dtype)
    if worst < -1e3:
        assert not bool(got["dg"][p["g"].cuda() == worst].any())


@pytest.mark.parametrize("Hg", [4, 2])
def test_gradients_equal_differences(Hg):
    """fp32, against differences of the kernel's own forward: the loss is linear in q and in v, so
    their differences have no error but rounding; k, g and h0 take a central one."""
    import gated_deltanet_chunked_02_amd as gdn
    p = make(1, 150, 4, Hg, 32, 24, "f32", seed=8)
    q = dev(p)
    got = run_bwd(p)

    def loss(**c):
        a = dict(q, **c)
        o, ht = gdn.linear_attention(a["q"], a["k"], a["v"], a["g"], initial_state=a["h0"])
        return (o.double() * q["do"].double()).sum() + (ht.double() * q["dht"].double()).sum()

    r = torch.Generator().manual_seed(9)
    for x in ("q", "k", "v", "g", "h0"):
        # along the gradient, where the difference is largest beside the rounding of the loss
        d = got["d" + x] / got["d" + x].norm()
        eps = 1e-2
        want = float(loss(**{x: q[x] + eps * d}) - loss(**{x: q[x] - eps * d})) / (2 * eps)
        have = float(got["d" + x].double().norm())
        # the third order of a step of 1e-2 along g (exp) is (1e-2)^2 / 6 of the first; the loss's
        # rounding is 1e-6 of its terms' sum over a difference of 2e-2 times the gradient's norm
        assert abs(want - have) <= 2e-3 * have, x


def test_strided_inputs_and_no_dg():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 70, 4, 2, 40, 24, "bf16", seed=11)
    q = dev(p)
    proj = torch.cat([q["q"].flatten(2), q["k"].flatten(2), q["v"].flatten(2)], -1)
    views = (proj[..., :80].unflatten(-1, (2, 40)), proj[..., 80:160].unflatten(-1, (2, 40)),
             proj[..., 160:].unflatten(-1, (4, 24)))
    a = run_bwd(p)
    wide = torch.zeros(2, 70, 4, 25, dtype=torch.bfloat16, device="cuda")
    wide[..., 1:] = q["do"]
    b = gdn.linear_attention_bwd(*views, q["g"], wide[..., 1:], dht=q["dht"],
                                 initial_state=q["h0"], need_dg=False)
    assert b[3] is None
    for x, t in zip(NAMES, b):
        assert t is None or torch.equal(a[x], t), x


@pytest.mark.parametrize("Hg", [4, 2])
@pytest.mark.parametrize("head", [False, True])
def test_gradients_of_no_sequence_are_left_alone(Hg, head):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(H=4, Hg=Hg, Dk=64, Dv=64, dtype="bf16", head=head, lens=[70, 200], seed=1)
    q = dev(p)
    wide = lambda t: torch.cat([t, torch.full_like(t[:, :37], float("nan"))], 1)  # noqa: E731
    desc = gdn.GdnLinearDesc(1, 307, 2, 4, Hg, 64, 64, 1, int(head), 0, 0.125, 0, 0, 0, None, 0)
    ws = torch.empty(gdn.gdn_linear_attn_bwd_workspace_size(desc), dtype=torch.uint8,
                     device="cuda")
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
    full = lambda *s, dt=torch.bfloat16: torch.full(s, 5.0, dtype=dt, device="cuda")  # noqa: E731
    out = dict(dq=full(1, 307, Hg, 64), dk=full(1, 307, Hg, 64), dv=full(1, 307, 4, 64),
               dg=full(4, dt=torch.float32) if head else full(1, 307, 4, dt=torch.float32),
               dh0=full(2, 4, 64, 64, dt=torch.float32))
    g = q["g"] if head else wide(q["g"])
    assert gdn.gdn_linear_attn_bwd(desc, wide(q["q"]), wide(q["k"]), wide(q["v"]), g, q["h0"],
                                   q["cu"], wide(q["do"]), q["dht"], *out.values()) == 0
    tokens = {x: t for x, t in out.items() if t.dim() > 1 and t.shape[1] == 307}
    for x, t in tokens.items():
        assert bool((t[:, 270:] == 5.0).all()), x
        out[x] = t[:, :270]
    check_all(p, out, oracle_bwd(p), "bf16")


def test_no_tokens():
    p = make(2, 0, 4, 2, 64, 40, seed=1)
    got = run_bwd(p)
    assert torch.equal(got["dh0"].cpu(), p["dht"]) and got["dq"].shape == (2, 0, 2, 64)
    p = make(2, 0, 4, 2, 64, 40, head=True, seed=1)
    got = run_bwd(p, dht=False)
    assert not bool(got["dh0"].any()) and not bool(got["dg"].any())


def test_reruns_are_equal_bit_for_bit():
    p = make(2, 700, 6, 2, 128, 64, "bf16", seed=5)
    a, b = run_bwd(p), run_bwd(p)
    for x in NAMES:
        assert torch.equal(a[x], b[x]), x


@pytest.mark.parametrize("H", [4, 130])
def test_replayed_from_a_graph(H):
    """Forward, step and gradient captured once and replayed on changed inputs give the eager calls'
    bits, with eager work and synchronisations between the replays."""
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 300, H, 2, 64, 64, "bf16", seed=7)
    q = dev(p)

    def run():
        args = (q["q"], q["k"], q["v"], q["g"])
        o, ht = gdn.linear_attention(*args, initial_state=q["h0"])
        last = gdn.linear_state_update(ht, *(t[:, 0] for t in args))
        grads = gdn.linear_attention_bwd(*args, q["do"], dht=q["dht"], initial_state=q["h0"])
        return [o, ht, last, *grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(3):
        for x in ("q", "v", "do"):
            q[x].copy_(torch.randn(q[x].shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_rows_past_2_to_31_elements():
    """A packed batch whose last sequences lie past 2^31 elements of q, k and v."""
    import gated_deltanet_chunked_02_amd as gdn
    H, D, lens = 128, 128, [131072, 130, 70]
    T = sum(lens)
    r = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=r, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, do = (n(1, T, H, D) for _ in range(4))
    g = -torch.rand(1, T, H, generator=r, device="cuda")
    cu = torch.tensor([0, 131072, 131202, T], dtype=torch.int32, device="cuda")
    assert q.numel() > 2 ** 31
    o, ht = gdn.linear_attention(q, k, v, g, cu_seqlens=cu)
    grads = gdn.linear_attention_bwd(q, k, v, g, do, cu_seqlens=cu)
    torch.cuda.synchronize()
    end = slice(131072, T)
    cut = [t[:, end].contiguous() for t in (q, k, v, g)]
    o2, ht2 = gdn.linear_attention(*cut, cu_seqlens=cu[1:] - 131072)
    grads2 = gdn.linear_attention_bwd(*cut, do[:, end].contiguous(), cu_seqlens=cu[1:] - 131072)
    # the two are split into other segments: fp32 roundings of states, and bf16 outputs that fall
    # to the other side of a half
    check("o", o[:, end], host(o2), 1e-4)
    check("ht", ht[1:], host(ht2), 1e-5)
    for x, a, b in zip(NAMES, grads, grads2):
        if b is not None:
            check(x, a[:, end], host(b), 2e-5 if x == "dg" else 1e-4)
