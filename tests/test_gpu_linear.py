"""GPU parity of linear attention (prompts and single tokens) against the fp64 oracle.

Tolerances, relative L2 over each tensor.  fp32 results: an output is a sum of at most 256 + 64
products in fp32, off by a rounding (2^-24) for each addition on a random walk, 18 x 2^-24 = 1.1e-6;
a state is remembered for at most about 20 chunks by these decays, sqrt(20) times that, 5e-6: 1e-5.
bf16 outputs: on each path one tensor is rounded to bf16, and then the output: two roundings of at
most 2^-8 each, 2 x 2^-8 + 1e-5.  States stay fp32 results whatever the type.  The same inputs
(already rounded to the dtype) go to both sides.
"""
import numpy as np
import pytest
import torch

from oracle import linear

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL_F32 = 1e-5
TOL = {"f32": TOL_F32, "bf16": 2 * 2.0 ** -8 + 1e-5}


def make(B=1, T=16, H=2, Hg=None, Dk=64, Dv=64, dtype="f32", head=False, h0=True, lens=None, seed=0):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    dt, Hg = DTYPES[dtype], Hg or H
    if lens is not None:
        B, T = 1, sum(lens)
    N = B if lens is None else len(lens)
    g = -torch.exp2(-8 * (torch.arange(H) + 1.0) / H) if head else \
        torch.nn.functional.logsigmoid(n(B, T, H) + 3)
    return dict(q=n(B, T, Hg, Dk).to(dt), k=n(B, T, Hg, Dk).to(dt), v=n(B, T, H, Dv).to(dt), g=g,
                h0=n(N, H, Dk, Dv) if h0 else None, do=n(B, T, H, Dv).to(dt),
                dht=n(N, H, Dk, Dv) * 0.1,
                cu=None if lens is None else torch.tensor(np.cumsum([0] + lens), dtype=torch.int32))


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def spans(p):
    return None if p["cu"] is None else p["cu"].numpy()


def oracle_fwd(p, scale=None):
    return linear.attention(*(host(p[x]) for x in ("q", "k", "v", "g")),
                            scale=p["q"].shape[-1] ** -0.5 if scale is None else scale,
                            h0=host(p["h0"]), cu=spans(p))


def dev(p):
    return {x: None if t is None else t.cuda() for x, t in p.items()}


def run_fwd(p, **kw):
    import gated_deltanet_chunked_02_amd as gdn
    q = dev(p)
    o, ht = gdn.linear_attention(q["q"], q["k"], q["v"], q["g"], initial_state=q["h0"],
                                 cu_seqlens=q["cu"], **kw)
    torch.cuda.synchronize()
    return o, ht


def check(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    if got.size:
        norm = np.linalg.norm(ref)
        e = np.linalg.norm(got - ref) / (norm if norm else 1.0)
        assert e <= tol, "%s: relative L2 %.3g over %.3g" % (name, e, tol)


def check_fwd(p, dtype, **kw):
    o_ref, ht_ref = oracle_fwd(p)
    o, ht = run_fwd(p, **kw)
    check("o", o, o_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


FWD = [
    # B, T, H, Hg, Dk, Dv, head, h0
    (1, 1, 1, 1, 8, 8, False, True),
    (1, 1, 2, 1, 64, 64, True, False),
    (2, 15, 3, 3, 64, 40, False, True),
    (2, 16, 4, 2, 16, 128, True, True),
    (1, 31, 2, 2, 96, 64, False, False),
    (1, 33, 2, 1, 128, 128, False, True),
    (3, 63, 5, 5, 40, 72, True, True),
    (1, 64, 2, 2, 64, 64, False, True),
    (1, 65, 6, 2, 128, 64, False, True),
    (2, 127, 4, 1, 64, 256, False, True),
    (1, 128, 2, 2, 256, 64, True, True),
    (1, 129, 2, 2, 192, 136, False, True),   # two segments, the second of one token
    (1, 200, 3, 1, 256, 256, False, False),
    (1, 700, 2, 1, 128, 128, False, True),
    (2, 300, 3, 3, 128, 96, True, True),
    (130, 3, 4, 4, 64, 64, False, True),     # more heads than run at once
    (5, 257, 64, 64, 32, 32, False, True),   # whole sequences of several chunks
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hg,Dk,Dv,head,h0", FWD)
def test_attention_matches_oracle(B, T, H, Hg, Dk, Dv, head, h0, dtype):
    check_fwd(make(B, T, H, Hg, Dk, Dv, dtype, head, h0, seed=B + T + Dk), dtype)


LENS = [[1], [5, 0, 1, 64, 65, 2], [0, 0, 7], [3, 500, 0, 129, 1, 63], [1] * 70, [0, 0],
        [128, 128, 128], [127, 129, 300]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H", [2, 96])  # segments, and twice the mean length
def test_packed_matches_oracle(lens, dtype, H):
    p = make(H=H, Hg=H // 2, Dk=16, Dv=32, dtype=dtype, lens=lens, seed=len(lens))
    o_ref, ht_ref = oracle_fwd(p)
    o, ht = run_fwd(p)
    check("o", o, o_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)
    for n, k in enumerate(lens):
        if k == 0:  # no tokens: the state passes through
            assert torch.equal(ht[n].cpu(), p["h0"][n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tokens_of_no_sequence_are_left_alone(dtype):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(H=4, Hg=2, Dk=64, Dv=64, dtype=dtype, lens=[70, 200], seed=1)
    q = dev(p)
    wide = lambda t: torch.cat([t, torch.full_like(t[:, :37], float("nan"))], 1)  # noqa: E731
    desc = gdn.GdnLinearDesc(1, 307, 2, 4, 2, 64, 64, 1 if dtype == "bf16" else 0, 0, 0, 0.125, 0,
                             0, 0, None, 0)
    ws = torch.empty(gdn.gdn_linear_attn_workspace_size(desc) + 1, dtype=torch.uint8, device="cuda")
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
    o = torch.full((1, 307, 4, 64), 5.0, dtype=DTYPES[dtype], device="cuda")
    ht = torch.empty(2, 4, 64, 64, device="cuda")
    assert gdn.gdn_linear_attn_fwd(desc, *(wide(q[x]) for x in ("q", "k", "v", "g")), q["h0"],
                                   q["cu"], o, ht) == 0
    assert bool((o[:, 270:] == 5.0).all())
    o_ref, ht_ref = oracle_fwd(p)
    check("o", o[:, :270], o_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("worst", [-60.0, -1e30, torch.finfo(torch.float32).min, -float("inf")])
def test_strong_decays(worst, dtype):
    """States forgotten altogether at some tokens; the decays after them keep their accuracy."""
    p = make(2, 150, 3, 3, 64, 64, dtype, seed=4)
    r = torch.rand(p["g"].shape, generator=torch.Generator().manual_seed(5))
    p["g"] = torch.where(r < 0.1, torch.tensor(worst), p["g"])
    p["g"][0, 70:75] = worst
    check_fwd(p, dtype)


def test_growing_states():
    """Positive log-decays, as long as the states fit fp32."""
    p = make(1, 100, 2, 2, 64, 64, seed=6)
    p["g"] = torch.rand(p["g"].shape, generator=torch.Generator().manual_seed(5)) * 0.2
    check_fwd(p, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_inputs_are_read_in_place(dtype):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 70, 4, 2, 40, 24, dtype, seed=11)
    q = dev(p)
    proj = torch.cat([q["q"].flatten(2), q["k"].flatten(2), q["v"].flatten(2)], -1)
    views = (proj[..., :80].unflatten(-1, (2, 40)), proj[..., 80:160].unflatten(-1, (2, 40)),
             proj[..., 160:].unflatten(-1, (4, 24)))
    o, ht = run_fwd(p)
    o2, ht2 = gdn.linear_attention(*views, q["g"], initial_state=q["h0"])
    assert torch.equal(o, o2) and torch.equal(ht, ht2)
    # rows at an odd address, heads in another order of axes, one k for every token: copied
    odd = torch.empty(proj.numel() + 1, dtype=proj.dtype, device="cuda")[1:].view(proj.shape)
    odd.copy_(proj)
    o3, ht3 = gdn.linear_attention(odd[..., :80].unflatten(-1, (2, 40)),
                                   q["k"].transpose(1, 2).contiguous().transpose(1, 2),
                                   odd[..., 160:].unflatten(-1, (4, 24)), q["g"],
                                   initial_state=q["h0"])
    assert torch.equal(o, o3) and torch.equal(ht, ht3)
    same = q["k"][:, :1].expand(2, 70, 2, 40)
    a = gdn.linear_attention(q["q"], same, q["v"], q["g"])
    b = gdn.linear_attention(q["q"], same.contiguous(), q["v"], q["g"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_scale_and_the_state_in_place():
    import gated_deltanet_chunked_02_amd as gdn
    for H in (2, 200):  # in segments and whole
        p = make(2, 400, H, 1, 32, 32, "f32", seed=12)
        q = dev(p)
        o_ref, ht_ref = oracle_fwd(p, scale=-1.5)
        desc = gdn.GdnLinearDesc(2, 400, 2, H, 1, 32, 32, 0, 0, 0, -1.5, 0, 0, 0, None, 0)
        ws = torch.empty(gdn.gdn_linear_attn_workspace_size(desc) + 1, dtype=torch.uint8,
                         device="cuda")
        desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel()
        o = torch.empty_like(q["v"])
        assert gdn.gdn_linear_attn_fwd(desc, q["q"], q["k"], q["v"], q["g"], q["h0"], None, o,
                                       q["h0"]) == 0
        check("o", o, o_ref, TOL_F32)
        check("ht", q["h0"], ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_head_and_sequence(dtype):
    p = make(H=4, Hg=2, Dk=64, Dv=64, dtype=dtype, lens=[100, 90, 200], seed=13)
    o0, ht0 = run_fwd(p)
    p["k"][0, 150, 0] = float("nan")   # sequence 1, value heads 0 and 1
    p["v"][0, 250, 3, 5] = float("inf")  # sequence 2, value head 3
    o, ht = run_fwd(p)
    for n, (a, e) in enumerate(((0, 100), (100, 190), (190, 390))):
        for h in range(4):
            if not (n == 1 and h < 2) and not (n == 2 and h == 3):
                assert torch.equal(o[0, a:e, h], o0[0, a:e, h])
                assert torch.equal(ht[n, h], ht0[n, h])
    assert bool(o[0, 150:190, :2].isnan().all()) and not bool(o[0, 250:, 3].isfinite().all())
    assert not bool(ht[2, 3].isfinite().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_tokens_equals_one_prompt(dtype):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(3, 160, 4, 2, 64, 40, dtype, seed=21)
    o_ref, ht_ref = oracle_fwd(p)
    q = dev(p)
    cut = lambda a, e: (q[x][:, a:e] for x in ("q", "k", "v", "g"))  # noqa: E731
    o, state = gdn.linear_attention(*cut(0, 150), initial_state=q["h0"])
    parts = [o]
    for t in range(150, 160):
        parts.append(gdn.linear_state_update(state, *(q[x][:, t] for x in ("q", "k", "v", "g")))
                     [:, None])
    check("o", torch.cat(parts, 1), o_ref, TOL[dtype])
    check("state", state, ht_ref, TOL_F32)


STEP = [
    # n, H, Hg, Dk, Dv, head
    (1, 1, 1, 8, 8, False),
    (1, 32, 16, 128, 128, False),
    (5, 6, 3, 40, 72, True),
    (3, 4, 1, 64, 64, False),
    (2, 3, 3, 256, 256, False),
    (2, 2, 1, 192, 24, True),
    (300, 2, 2, 16, 32, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,Hg,Dk,Dv,head", STEP)
def test_step_matches_oracle(n, H, Hg, Dk, Dv, head, dtype):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(n, 1, H, Hg, Dk, Dv, dtype, head, seed=n + Dk)
    o_ref, ht_ref = oracle_fwd(p)
    q = dev(p)
    pool = torch.full((2 * n + 2, H, Dk, Dv), 7.0, device="cuda")
    perm = torch.randperm(2 * n + 2, generator=torch.Generator().manual_seed(n)).cuda()
    read, write, rest = perm[:n], perm[n:2 * n], perm[2 * n:]
    pool[read] = q["h0"]
    before = pool.clone()
    o = gdn.linear_state_update(pool, q["q"][:, 0], q["k"][:, 0], q["v"][:, 0],
                                q["g"] if head else q["g"][:, 0], cache_indices=read,
                                out_indices=write)
    torch.cuda.synchronize()
    # one rounding, of the output
    check("o", o, o_ref[:, 0], TOL_F32 if dtype == "f32" else 2.0 ** -8 + 1e-5)
    check("states", pool[write], ht_ref, TOL_F32)
    assert torch.equal(pool[read], before[read]) and torch.equal(pool[rest], before[rest])


def test_step_lines_outside_the_pool():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(3, 1, 2, 2, 64, 64, seed=2)
    q = dev(p)
    pool = q["h0"].clone()
    idx = torch.tensor([-1, 1, 3], dtype=torch.int32, device="cuda")
    o = gdn.linear_state_update(pool, *(q[x][:, 0] for x in ("q", "k", "v", "g")),
                                cache_indices=idx)
    p["h0"] = p["h0"].clone()
    p["h0"][0], p["h0"][2] = 0, 0
    o_ref, ht_ref = oracle_fwd(p)
    check("o", o, o_ref[:, 0], TOL_F32)
    assert torch.equal(pool[0], q["h0"][0]) and torch.equal(pool[2], q["h0"][2])
    check("line 1", pool[1], ht_ref[1], TOL_F32)
    # -inf forgets the line
    g = torch.full((2,), -float("inf"), device="cuda")
    gdn.linear_state_update(pool, *(q[x][:, 0] for x in ("q", "k", "v")), g)
    want = q["k"][:, 0][..., None] * q["v"][:, 0][:, :, None]
    assert torch.equal(pool, want)


def test_step_of_strided_rows():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(4, 1, 4, 2, 64, 64, "bf16", seed=3)
    q = dev(p)
    proj = torch.cat([q[x][:, 0].flatten(1) for x in ("q", "k", "v")], -1)
    a, b = q["h0"].clone(), q["h0"].clone()
    o = gdn.linear_state_update(a, *(q[x][:, 0] for x in ("q", "k", "v", "g")))
    o2 = gdn.linear_state_update(b, proj[:, :128].unflatten(-1, (2, 64)),
                                 proj[:, 128:256].unflatten(-1, (2, 64)),
                                 proj[:, 256:].unflatten(-1, (4, 64)), q["g"][:, 0])
    assert torch.equal(o, o2) and torch.equal(a, b)


def test_no_tokens_and_no_sequences():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 0, 4, 2, 64, 40, seed=1)
    o, ht = run_fwd(p)
    assert o.shape == (2, 0, 4, 40) and torch.equal(ht.cpu(), p["h0"])
    p["h0"] = None
    assert not bool(run_fwd(p)[1].any())
    p = make(0, 5, 4, 2, 64, 40, h0=False)
    o, ht = run_fwd(p)
    assert o.shape == (0, 5, 4, 40) and ht.shape == (0, 4, 64, 40)
    q = dev(make(1, 5, 4, 2, 64, 40, h0=False))
    o, ht = gdn.linear_attention(q["q"], q["k"], q["v"], q["g"],
                                 cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert ht.shape == (0, 4, 64, 40)


def test_on_another_stream_with_a_given_workspace():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(1, 500, 2, 2, 64, 64, "bf16", seed=30)
    o0, ht0 = run_fwd(p)
    q = dev(p)
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o, ht = gdn.linear_attention(q["q"], q["k"], q["v"], q["g"], initial_state=q["h0"],
                                     workspace=ws)
        o2, none = gdn.linear_attention(q["q"], q["k"], q["v"], q["g"], initial_state=q["h0"],
                                        output_final_state=False)
    s.synchronize()
    assert torch.equal(o, o0) and torch.equal(ht, ht0) and torch.equal(o2, o0) and none is None
