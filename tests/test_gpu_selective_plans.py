"""The selective scan's ways of running a batch (whole sequences, chunks whose start states a launch
of its own composes, chunks that compose their own), each against the fp64 oracle and each with the
states carried in place.

Every case names the chunk slots it is meant for, which the workspace's size gives away (see
``slots_of``): 0 for whole sequences, else sequence by sequence its chunks (and one more a sequence of
a packed batch or of a batch of one, which may come as either, at most).  Tolerances, relative L2.  fp32: a state is a sum over its tokens, each rounded
twice, and over chunks whose decay's exponent is rounded once; rounding errors of unlike sign over the
at most 600 tokens here add up to about sqrt(1200) x 2^-24 = 2e-6 of it: 1e-5.  bf16 outputs: one
rounding to 8 significant bits more, 2^-8 + 1e-5.
"""
import pytest
import torch

from test_gpu_selective import TOL, TOL_F32, check, dev, make, oracle_fwd, run_fwd

pytestmark = pytest.mark.gpu


def desc_of(p):
    import gated_deltanet_chunked_02_amd as gdn
    B, T, C = p["x"].shape
    N = B if p["cu"] is None else p["cu"].numel() - 1
    return gdn.GdnScanDesc(B=B, T=T, N=N, channels=C, groups=p["B"].shape[2],
                           dstate=p["A"].shape[1], dtype=int(p["x"].dtype == torch.bfloat16),
                           dt_softplus=1)


def slots_of(d):
    """Chunk slots the forward plans: what its workspace holds beside the B and C rows."""
    import gated_deltanet_chunked_02_amd as gdn
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    rest = gdn.gdn_selective_scan_workspace_size(d)
    padded = next(n for n in (4, 8, 16, 32, 64, 128, 256) if n >= d.dstate)
    rest -= up(d.B * d.T * d.groups * 2 * padded * 4)
    slots = 0
    while up(slots * d.dstate * d.channels * 4) + up(slots * d.channels * 4) < rest:
        slots += 1
    return slots


def run_in_place(p, ht=None):
    """The raw call on one buffer for the initial and the final states (or on ``ht``)."""
    import gated_deltanet_chunked_02_amd as gdn
    q = dev(p)
    d = desc_of(p)
    ws = torch.empty(gdn.gdn_selective_scan_workspace_size(d), dtype=torch.uint8, device="cuda")
    d.workspace, d.workspace_bytes = ws.data_ptr(), ws.numel()
    y = torch.empty_like(q["x"])
    ht = q["h0"] if ht is None else ht
    st = gdn.gdn_selective_scan_fwd(d, q["x"], q["dt"], q["A"], q["B"], q["C"], q["D"], q["z"],
                                    q["dt_bias"], q["h0"], q["cu"], y, ht)
    torch.cuda.synchronize()
    assert st == 0
    return y, ht


@pytest.mark.parametrize("B,T,C,G,S,lens,slots", [
    (2, 60, 64, 1, 16, None, 0),      # whole sequences
    (1, 225, 64, 1, 16, None, 8),     # 8 chunks that compose their own start, the last of one token
    (1, 225, 64, 1, 4, None, 8),
    (2, 400, 50, 50, 16, None, 10),
    (1, 0, 64, 1, 16, [97, 1, 127], 10),
    (1, 500, 64, 1, 16, None, 16),    # chunks composed by a launch of their own
    (1, 225, 64, 1, 64, None, 8),
])
def test_states_in_place(B, T, C, G, S, lens, slots):
    """h0 and ht in one buffer: the same bits as in two."""
    p = make(B, T, C, G, S, "f32", lens=lens, seed=B + T + S)
    assert slots_of(desc_of(p)) == slots
    y2, ht2 = run_in_place(p, torch.empty_like(p["h0"], device="cuda"))
    y1, ht1 = run_in_place(p)
    assert torch.equal(y1, y2) and torch.equal(ht1, ht2)
    y_ref, ht_ref = oracle_fwd(p)
    check("y", y1, y_ref, TOL_F32)
    check("ht", ht1, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,G,S,h0,slots", [
    # a dense sequence whose chunks compose their own start states: 2 to 8 of them
    (1, 225, 64, 1, 16, True, 8), (1, 256, 64, 1, 16, True, 9), (1, 256, 64, 1, 16, False, 9),
    (1, 225, 64, 1, 4, True, 8), (1, 250, 70, 2, 3, False, 8),
    (1, 225, 64, 1, 8, True, 8), (1, 193, 130, 1, 7, True, 7),
    (2, 225, 64, 1, 16, True, 16), (2, 256, 100, 1, 8, True, 16), (2, 400, 50, 50, 16, False, 10),
    (1, 600, 80, 80, 16, True, 6), (2, 300, 80, 80, 16, True, 6), (1, 400, 170, 170, 9, True, 3),
    (2, 200, 200, 200, 2, True, 6),
    # composed by a launch of their own: many chunks, or more states than 16
    (1, 300, 64, 1, 4, True, 10), (1, 300, 65, 1, 8, False, 10), (1, 577, 64, 1, 16, True, 19),
    (1, 225, 64, 1, 17, True, 8), (1, 300, 64, 1, 32, True, 10), (2, 225, 70, 1, 32, False, 16),
    (1, 225, 64, 1, 65, True, 8), (1, 300, 64, 1, 128, True, 10), (2, 193, 40, 2, 128, False, 14),
    (1, 225, 64, 1, 129, True, 8), (1, 300, 64, 1, 256, False, 10), (2, 225, 30, 1, 256, True, 16),
])
def test_dense_chunks(B, T, C, G, S, h0, slots, dtype):
    p = make(B, T, C, G, S, dtype, h0=h0, seed=B + T + C + S)
    assert slots_of(desc_of(p)) == slots
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens,slots", [([97, 1, 0, 127], 11),        # at most 8 chunks by length
                                        ([3, 290, 0, 129, 1, 63], 21)])
def test_packed_chunks(lens, slots, S, dtype):
    p = make(C=72, G=2, S=S, dtype=dtype, lens=lens, seed=S)
    assert slots_of(desc_of(p)) == slots
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [1, 4, 8, 32, 33, 256])
def test_packed_gradients(S, dtype):
    """Every number of waves, and one state block (up to 32 states) or several."""
    from test_gpu_selective_bwd import check_all, oracle_bwd, run_bwd
    p = make(C=72, G=2, S=S, dtype=dtype, lens=[3, 200, 0, 129, 1, 63], seed=S)
    check_all(p, run_bwd(p), oracle_bwd(p), dtype)


def test_rows_far_apart():
    """One token of a long batch, 8 MB from row to row, and a prompt whose rows are 256 MB apart: the
    same bits as from rows one after another."""
    import gated_deltanet_chunked_02_amd as gdn
    p = make(4, 1, 4096, 1, 16, "bf16", seed=3)
    q = dev(p)
    wide = torch.zeros(4, 1024, 4096, dtype=torch.bfloat16, device="cuda")
    at = wide[:, 700:701]
    at.copy_(q["x"])
    kw = dict(D=q["D"], z=q["z"], dt_bias=q["dt_bias"], dt_softplus=True)
    one = lambda t: t[:, 0]  # noqa: E731
    kw1 = dict(kw, z=one(q["z"]))
    rest = (q["dt"], q["A"], q["B"], q["C"])
    rest1 = tuple(t if t is q["A"] else one(t) for t in rest)
    a, b = q["h0"].clone(), q["h0"].clone()
    assert torch.equal(gdn.selective_state_update(a, one(at), *rest1, **kw1),
                       gdn.selective_state_update(b, one(q["x"]), *rest1, **kw1))
    assert torch.equal(a, b)
    for got, want in zip(gdn.selective_scan(at, *rest, initial_state=q["h0"], **kw),
                         gdn.selective_scan(q["x"], *rest, initial_state=q["h0"], **kw)):
        assert torch.equal(got, want)
    for got, want in zip(gdn.selective_scan_bwd(at, *rest, q["dy"], dht=q["dht"], **kw),
                         gdn.selective_scan_bwd(q["x"], *rest, q["dy"], dht=q["dht"], **kw)):
        assert got is None and want is None or torch.equal(got, want)
    del wide
    p = make(1, 3, 64, 1, 16, "f32", seed=4)
    q = dev(p)
    far = torch.zeros(1, 3, 1 << 26, device="cuda")[..., 5:69]
    far.copy_(q["x"])
    rest = (q["dt"], q["A"], q["B"], q["C"])
    kw = dict(D=q["D"], z=q["z"], dt_bias=q["dt_bias"], dt_softplus=True, initial_state=q["h0"])
    y, ht = gdn.selective_scan(far, *rest, **kw)
    y_ref, ht_ref = oracle_fwd(p)
    check("y", y, y_ref, TOL_F32)
    check("ht", ht, ht_ref, TOL_F32)
    for got, want in zip(gdn.selective_scan_bwd(far, *rest, q["dy"], **kw),
                         gdn.selective_scan_bwd(q["x"], *rest, q["dy"], **kw)):
        assert torch.equal(got, want)


def test_many_groups():
    """A group for each of 70000 channels: more blocks of channels than 16 bits count."""
    import gated_deltanet_chunked_02_amd as gdn
    from test_gpu_selective_bwd import check_all, oracle_bwd, run_bwd
    p = make(2, 5, 70000, 70000, 1, "f32", seed=8)
    y_ref, ht_ref = oracle_fwd(p)
    y, ht = run_fwd(p)
    check("y", y, y_ref, TOL_F32)
    check("ht", ht, ht_ref, TOL_F32)
    check_all(p, run_bwd(p), oracle_bwd(p), "f32")
    p = make(2, 1, 70000, 70000, 1, "f32", seed=9)
    q = dev(p)
    one = [q[k] if k == "A" else q[k][:, 0] for k in ("x", "dt", "A", "B", "C")]
    y = gdn.selective_state_update(q["h0"], *one, D=q["D"], z=q["z"][:, 0], dt_bias=q["dt_bias"],
                                   dt_softplus=True)
    y_ref, ht_ref = oracle_fwd(p)
    check("y", y, y_ref[:, 0], TOL_F32)
    check("state", q["h0"], ht_ref, TOL_F32)
