"""GPU parity of the selective scan (prompts and single tokens) against the fp64 oracle.

Tolerances, relative L2 over each tensor.  fp32: a state carries the rounding of the decays it
went through; with the decays of these inputs it remembers at most about 64 tokens, each with
one rounding of the exponent and one of the update, 64 x 2^-23 = 8e-6: 1e-5.  bf16 outputs: one
rounding to 8 significant bits, at most 2^-8 of each value: 2^-8 + 1e-5.  The same inputs (already rounded to the
dtype) go to both sides.
"""
import numpy as np
import pytest
import torch

from oracle import selective

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL_F32 = 1e-5
TOL = {"f32": TOL_F32, "bf16": 2.0 ** -8 + 1e-5}


def make(B=1, T=16, C=64, G=1, S=16, dtype="f32", z=True, h0=True, D=True, bias=True, lens=None,
         seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DTYPES[dtype]
    if lens is not None:
        B, T = 1, sum(lens)
    N = B if lens is None else len(lens)
    first = torch.exp(torch.rand(C, generator=g) * np.log(100.0) + np.log(1e-3))
    p = dict(x=n(B, T, C).to(dt), dt=(n(B, T, C) * 0.5).to(dt),
             A=-torch.arange(1, S + 1).float() * torch.exp(0.2 * n(C, S)),
             B=n(B, T, G, S).to(dt), C=n(B, T, G, S).to(dt), D=n(C) if D else None,
             z=n(B, T, C).to(dt) if z else None,
             dt_bias=(first + torch.log(-torch.expm1(-first))) if bias else None,
             h0=n(N, C, S) * 0.5 if h0 else None,
             cu=None if lens is None else torch.tensor(np.cumsum([0] + lens), dtype=torch.int32))
    p["dy"] = n(B, T, C).to(dt)
    p["dht"] = n(N, C, S) * 0.5
    return p


def host(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def oracle_fwd(p, softplus=True):
    return selective.scan(*(host(p[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")),
                          dt_softplus=softplus, h0=host(p["h0"]),
                          cu=None if p["cu"] is None else p["cu"].numpy())


def dev(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def run_fwd(p, softplus=True, **kw):
    import gated_deltanet_chunked_02_amd as gdn
    q = dev(p)
    y, ht = gdn.selective_scan(q["x"], q["dt"], q["A"], q["B"], q["C"], D=q["D"], z=q["z"],
                               dt_bias=q["dt_bias"], dt_softplus=softplus,
                               initial_state=q["h0"], cu_seqlens=q["cu"], **kw)
    torch.cuda.synchronize()
    return y, ht


def rel(a, ref):
    a, ref = np.asarray(a, np.float64), np.asarray(ref, np.float64)
    d = np.linalg.norm(ref)
    return float(np.linalg.norm(a - ref) / (d if d else 1.0))


def check(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    if got.size:
        e = rel(got, ref)
        assert e <= tol, "%s: relative L2 %.3g over %.3g" % (name, e, tol)


FWD = [
    # B, T, C, G, S, dtype, z, h0
    (1, 1, 1, 1, 1, "f32", True, True),
    (1, 1, 64, 1, 16, "bf16", False, True),
    (2, 15, 63, 1, 16, "f32", True, True),
    (2, 16, 65, 1, 16, "bf16", True, False),
    (3, 17, 200, 4, 16, "f32", False, False),
    (1, 33, 130, 130, 4, "f32", True, True),   # a group for every channel
    (2, 40, 96, 3, 5, "bf16", True, True),
    (1, 70, 64, 2, 8, "f32", True, True),
    (1, 300, 64, 1, 16, "f32", True, True),    # several chunks
    (1, 1000, 70, 1, 16, "bf16", True, True),
    (1, 129, 100, 1, 3, "f32", True, True),
    (1, 140, 48, 1, 17, "f32", True, True),
    (2, 90, 64, 2, 32, "bf16", True, True),
    (1, 200, 64, 1, 64, "f32", False, True),
    (1, 100, 40, 1, 100, "f32", True, True),
    (1, 80, 24, 1, 256, "f32", True, True),
    (70, 3, 64, 1, 16, "f32", True, True),
]


@pytest.mark.parametrize("B,T,C,G,S,dtype,z,h0", FWD)
def test_scan_matches_oracle(B, T, C, G, S, dtype, z, h0):
    p = make(B, T, C, G, S, dtype, z, h0, seed=B + T + C + S)
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [5, 0, 1, 64, 65, 2], [0, 0, 7], [3, 500, 0, 129, 1, 63],
                                  [1] * 70, [0, 0]])
def test_packed_matches_oracle(lens, dtype):
    p = make(C=72, G=2, S=16, dtype=dtype, lens=lens, seed=len(lens))
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)
    for n, k in enumerate(lens):
        if k == 0:  # no tokens: the state passes through
            assert torch.equal(ht[n].cpu(), p["h0"][n])


@pytest.mark.parametrize("B,T,C,G,S,dtype", [
    (1, 31, 64, 1, 16, "f32"), (1, 32, 64, 1, 16, "bf16"), (1, 63, 64, 1, 16, "f32"),
    (1, 64, 64, 1, 16, "bf16"), (1, 65, 65, 1, 16, "f32"), (2, 97, 64, 1, 8, "f32"),
    (2, 100, 130, 130, 16, "f32"),   # blocks enough for whole sequences
    (1, 90, 200, 200, 4, "bf16"),
    (1, 70, 190, 95, 256, "f32"),
    (1, 400, 50, 50, 16, "f32"),     # chunks of 48 tokens
    (3, 200, 40, 40, 64, "f32"),
])
def test_chunk_lengths(B, T, C, G, S, dtype):
    """Lengths about a chunk's, whole sequences and longer chunks (a group has its own channel
    blocks, so many groups of few channels make many workgroups)."""
    p = make(B, T, C, G, S, dtype, seed=B + T + C + S)
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_of_many_blocks_matches_oracle(dtype):
    """Sequences split at twice their mean length."""
    p = make(C=104, G=104, S=16, dtype=dtype, lens=[3, 500, 0, 129, 1, 63], seed=2)
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


def test_without_softplus_bias_or_skip():
    p = make(2, 50, 64, 1, 16, D=False, bias=False, seed=9)
    p["dt"] = torch.rand(p["dt"].shape, generator=torch.Generator().manual_seed(1)) * 0.1
    y_ref, ht_ref = oracle_fwd(p, softplus=False)
    y, ht = run_fwd(p, softplus=False)
    check("y", y, y_ref, TOL_F32)
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_far_from_zero(dtype):
    """dt from -60 to 60: steps that vanish and steps whose decay underflows to zero."""
    p = make(1, 80, 64, 1, 16, dtype, bias=False, seed=4)
    p["dt"] = torch.linspace(-60, 60, 80)[None, :, None].expand(1, 80, 64).to(DTYPES[dtype])
    p["dt"] = p["dt"].contiguous()
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_inputs_are_read_in_place(dtype):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 70, 65, 1, 7, dtype, seed=11)
    q = dev(p)
    wide = torch.zeros(2, 70, 65 * 3 + 1, dtype=DTYPES[dtype], device="cuda")
    views = {}
    for i, k in enumerate(("x", "dt", "z")):
        views[k] = wide[..., 1 + 65 * i:1 + 65 * (i + 1)]
        views[k].copy_(q[k])
    proj = torch.zeros(2, 70, 5 + 14, dtype=DTYPES[dtype], device="cuda")
    proj[..., 5:12], proj[..., 12:] = q["B"][:, :, 0], q["C"][:, :, 0]
    views["B"], views["C"] = proj[..., 5:12].unflatten(-1, (1, 7)), proj[..., 12:].unflatten(-1, (1, 7))
    y, ht = gdn.selective_scan(views["x"], views["dt"], q["A"], views["B"], views["C"], D=q["D"],
                               z=views["z"], dt_bias=q["dt_bias"], dt_softplus=True,
                               initial_state=q["h0"])
    y2, ht2 = run_fwd(p)
    assert torch.equal(y, y2) and torch.equal(ht, ht2)
    # axes in another order, and a broadcast gate: copied, same answer
    y3, _ = gdn.selective_scan(q["x"].transpose(0, 1).contiguous().transpose(0, 1), q["dt"],
                               q["A"], q["B"], q["C"], D=q["D"],
                               z=q["z"][:, :1].expand(2, 70, 65), dt_bias=q["dt_bias"],
                               dt_softplus=True, initial_state=q["h0"])
    y4, _ = gdn.selective_scan(q["x"], q["dt"], q["A"], q["B"], q["C"], D=q["D"],
                               z=q["z"][:, :1].expand(2, 70, 65).contiguous(),
                               dt_bias=q["dt_bias"], dt_softplus=True, initial_state=q["h0"])
    assert torch.equal(y3, y4)


def test_prompt_then_tokens_equals_one_prompt():
    """A prompt, then one token a call with the state carried in place, equals one call over all
    tokens to fp32 rounding of the states."""
    import gated_deltanet_chunked_02_amd as gdn
    p = make(3, 40, 100, 2, 16, "f32", seed=21)
    y_ref, ht_ref = oracle_fwd(p)
    q = dev(p)
    cut = lambda a, b: [q[k][:, a:b] for k in ("x", "dt")]  # noqa: E731
    kw = dict(D=q["D"], dt_bias=q["dt_bias"], dt_softplus=True)
    x, dt = cut(0, 33)
    y0, state = gdn.selective_scan(x, dt, q["A"], q["B"][:, :33], q["C"][:, :33],
                                   z=q["z"][:, :33], initial_state=q["h0"], **kw)
    ys = [y0]
    for t in range(33, 40):
        ys.append(gdn.selective_state_update(state, q["x"][:, t], q["dt"][:, t], q["A"],
                                             q["B"][:, t], q["C"][:, t], z=q["z"][:, t],
                                             **kw)[:, None])
    check("y", torch.cat(ys, 1), y_ref, TOL_F32)
    check("state", state, ht_ref, TOL_F32)


STEP = [
    # n, C, G, S, dtype, z
    (1, 1, 1, 1, "f32", True),
    (1, 4096, 1, 16, "bf16", True),
    (5, 100, 4, 16, "f32", True),
    (3, 70, 1, 12, "bf16", False),
    (2, 33, 33, 4, "f32", True),
    (4, 65, 1, 5, "bf16", True),
    (7, 128, 2, 64, "f32", False),
    (2, 96, 1, 128, "bf16", True),
    (2, 30, 1, 256, "f32", True),
    (300, 64, 1, 8, "bf16", True),
]


@pytest.mark.parametrize("n,C,G,S,dtype,z", STEP)
def test_step_matches_oracle(n, C, G, S, dtype, z):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(n, 1, C, G, S, dtype, z, seed=n + C + S)
    y_ref, ht_ref = oracle_fwd(p)
    q = dev(p)
    pool = torch.full((2 * n + 2, C, S), 7.0, device="cuda")
    perm = torch.randperm(2 * n + 2, generator=torch.Generator().manual_seed(n))
    read, write = perm[:n].cuda(), perm[n:2 * n].cuda()
    pool[read] = q["h0"]
    before = pool.clone()
    y = gdn.selective_state_update(pool, q["x"][:, 0], q["dt"][:, 0], q["A"], q["B"][:, 0],
                                   q["C"][:, 0], D=q["D"], z=q["z"][:, 0] if z else None,
                                   dt_bias=q["dt_bias"], dt_softplus=True, cache_indices=read,
                                   out_indices=write)
    torch.cuda.synchronize()
    check("y", y, y_ref[:, 0], TOL[dtype])
    check("states", pool[write], ht_ref, TOL_F32)
    rest = perm[2 * n:].cuda()
    assert torch.equal(pool[read], before[read]) and torch.equal(pool[rest], before[rest])


def test_step_lines_outside_the_pool():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(3, 1, 64, 1, 16, seed=2)
    q = dev(p)
    args = [q["x"][:, 0], q["dt"][:, 0], q["A"], q["B"][:, 0], q["C"][:, 0]]
    pool = q["h0"].clone()
    idx = torch.tensor([-1, 1, 3], dtype=torch.int32, device="cuda")
    y = gdn.selective_state_update(pool, *args, dt_softplus=True, cache_indices=idx)
    p0 = dict(p, h0=p["h0"].clone(), D=None, z=None, dt_bias=None)
    p0["h0"][0], p0["h0"][2] = 0, 0
    y_ref, ht_ref = oracle_fwd(p0)
    check("y", y, y_ref[:, 0], TOL_F32)
    assert torch.equal(pool[0], q["h0"][0]) and torch.equal(pool[2], q["h0"][2])
    check("line 1", pool[1], ht_ref[1], TOL_F32)


def test_step_on_unaligned_rows():
    """State and A that begin 4 bytes past a 16-byte boundary, strided rows."""
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 1, 64, 1, 8, seed=6)
    q = dev(p)
    flat = torch.zeros(2 * 64 * 8 + 1, device="cuda")[1:]
    state = flat.view(2, 64, 8)
    state.copy_(q["h0"])
    A = torch.zeros(64 * 8 + 1, device="cuda")[1:].view(64, 8)
    A.copy_(q["A"])
    wide = torch.zeros(2, 129, device="cuda")
    wide[:, 65:] = q["x"][:, 0]
    kw = dict(D=q["D"], z=q["z"][:, 0], dt_bias=q["dt_bias"], dt_softplus=True)
    y = gdn.selective_state_update(state, wide[:, 65:], q["dt"][:, 0], A, q["B"][:, 0],
                                   q["C"][:, 0], **kw)
    y_ref, ht_ref = oracle_fwd(p)
    check("y", y, y_ref[:, 0], TOL_F32)
    check("state", state, ht_ref, TOL_F32)


def test_on_another_stream():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(1, 500, 64, 1, 16, seed=30)
    y0, ht0 = run_fwd(p)
    q = dev(p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, ht = gdn.selective_scan(q["x"], q["dt"], q["A"], q["B"], q["C"], D=q["D"], z=q["z"],
                                   dt_bias=q["dt_bias"], dt_softplus=True,
                                   initial_state=q["h0"])
    s.synchronize()
    assert torch.equal(y, y0) and torch.equal(ht, ht0)


def test_given_workspace_and_final_state_left_out():
    p = make(1, 500, 64, 1, 16, seed=31)
    y0, _ = run_fwd(p)
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    y, ht = run_fwd(p, output_final_state=False, workspace=ws)
    assert ht is None and torch.equal(y, y0)
