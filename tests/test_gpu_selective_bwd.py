"""GPU parity of the selective scan's gradient against the fp64 oracle's.

Tolerances, relative L2 over each tensor.  fp32: states and gradients each carry at most 8e-6 of
their decays' rounding (see test_gpu_selective), a gradient is a product of both, 1.6e-5, and sums
over tokens or channels add errors no faster than the terms: 2e-5.  bf16 outputs: one rounding to
8 significant bits more, 2^-8 + 2e-5.
"""
import pytest
import torch

from oracle import selective
from test_gpu_selective import check, dev, host, make

pytestmark = pytest.mark.gpu

TOL_F32 = 2e-5
TOL = {"f32": TOL_F32, "bf16": 2.0 ** -8 + 2e-5}
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")


def oracle_bwd(p, softplus=True, dht=True):
    return selective.scan_backward(
        *(host(p[k]) for k in ("x", "dt", "A", "B", "C", "dy", "D", "z", "dt_bias")),
        dt_softplus=softplus, h0=host(p["h0"]), dht=host(p["dht"]) if dht else None,
        cu=None if p["cu"] is None else p["cu"].numpy())


def run_bwd(p, softplus=True, dht=True, **kw):
    import gated_deltanet_chunked_02_amd as gdn
    q = dev(p)
    out = gdn.selective_scan_bwd(q["x"], q["dt"], q["A"], q["B"], q["C"], q["dy"], D=q["D"],
                                 z=q["z"], dt_bias=q["dt_bias"], dt_softplus=softplus,
                                 initial_state=q["h0"], dht=q["dht"] if dht else None,
                                 cu_seqlens=q["cu"], **kw)
    torch.cuda.synchronize()
    return dict(zip(NAMES, out))


def check_all(p, got, ref, dtype):
    given = dict(dD="D", dz="z", dbias="dt_bias", dh0="h0")
    for k in NAMES:
        if k in given and p[given[k]] is None:
            assert got[k] is None, k
        else:
            check(k, got[k], ref[k], TOL_F32 if k in ("dA", "dD", "dbias", "dh0") else TOL[dtype])


BWD = [
    # B, T, C, G, S, dtype, z, h0, dht
    (1, 1, 1, 1, 1, "f32", True, True, True),
    (1, 1, 64, 1, 16, "bf16", False, True, True),
    (2, 7, 63, 1, 16, "f32", True, True, False),
    (2, 8, 65, 1, 16, "bf16", True, False, True),
    (3, 9, 200, 4, 16, "f32", False, False, False),
    (1, 33, 130, 130, 4, "f32", True, True, True),   # a group for every channel
    (2, 40, 96, 3, 5, "bf16", True, True, True),
    (1, 64, 64, 2, 8, "f32", True, True, True),
    (1, 65, 64, 1, 16, "f32", True, True, True),     # two chunks, the second of one token
    (2, 200, 70, 1, 16, "bf16", True, True, True),
    (1, 300, 64, 1, 16, "f32", False, True, True),
    (1, 129, 100, 1, 3, "f32", True, True, True),
    (1, 140, 48, 1, 17, "f32", True, True, True),    # two state blocks, the second of one
    (2, 90, 64, 2, 32, "bf16", True, True, True),
    (1, 100, 40, 1, 100, "f32", True, True, True),
    (1, 70, 24, 1, 256, "f32", True, True, True),
    (70, 3, 64, 1, 16, "f32", True, True, True),
]


@pytest.mark.parametrize("B,T,C,G,S,dtype,z,h0,dht", BWD)
def test_gradients_match_oracle(B, T, C, G, S, dtype, z, h0, dht):
    p = make(B, T, C, G, S, dtype, z, h0, seed=B + T + C + S)
    check_all(p, run_bwd(p, dht=dht), oracle_bwd(p, dht=dht), dtype)


@pytest.mark.parametrize("B,T,C,G,S,dtype", [
    (1, 16, 64, 1, 16, "f32"), (1, 17, 64, 1, 16, "bf16"), (1, 31, 64, 1, 4, "f32"),
    (1, 130, 128, 64, 16, "f32"),    # chunks of 32 tokens
    (1, 330, 128, 64, 16, "f32"),    # of 64
    (2, 129, 128, 64, 16, "bf16"),
    (1, 650, 128, 64, 8, "bf16"),
    (1, 140, 128, 64, 40, "f32"),    # and two blocks of states
    (1, 1100, 128, 64, 2, "f32"),
])
def test_chunk_lengths(B, T, C, G, S, dtype):
    """Chunks of every length that the number of workgroups chooses (a group has its own channel
    blocks, so many groups of few channels make many workgroups)."""
    p = make(B, T, C, G, S, dtype, seed=B + T + C + S)
    check_all(p, run_bwd(p), oracle_bwd(p), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_gradients_of_many_blocks_match_oracle(dtype):
    p = make(C=128, G=64, S=16, dtype=dtype, lens=[3, 200, 0, 129, 1, 63], seed=2)
    check_all(p, run_bwd(p), oracle_bwd(p), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [5, 0, 1, 64, 65, 2], [0, 0, 7], [3, 300, 0, 129, 1, 63],
                                  [1] * 70, [0, 0]])
def test_packed_gradients_match_oracle(lens, dtype):
    p = make(C=72, G=2, S=16, dtype=dtype, lens=lens, seed=len(lens))
    got = run_bwd(p)
    check_all(p, got, oracle_bwd(p), dtype)
    for n, k in enumerate(lens):
        if k == 0:  # no tokens: the gradient passes through
            assert torch.equal(got["dh0"][n].cpu(), p["dht"][n])


def test_without_softplus_bias_or_skip():
    p = make(2, 50, 64, 1, 16, D=False, bias=False, seed=9)
    p["dt"] = torch.rand(p["dt"].shape, generator=torch.Generator().manual_seed(1)) * 0.1
    check_all(p, run_bwd(p, softplus=False), oracle_bwd(p, softplus=False), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_far_from_zero(dtype):
    """dt from -60 to 60: steps that vanish and steps whose decay underflows to zero."""
    p = make(1, 80, 64, 1, 16, dtype, bias=False, seed=4)
    p["dt"] = torch.linspace(-60, 60, 80)[None, :, None].expand(1, 80, 64).to(p["x"].dtype)
    p["dt"] = p["dt"].contiguous()
    check_all(p, run_bwd(p), oracle_bwd(p), dtype)


def test_gradients_against_differences_of_the_forward():
    """The directional derivative from the gradients against differences of the library's own
    forward along one random direction, fp32: with a step of 2^-7 and the loss in fp64 the
    differences' error is (2^-7)^2 of third derivatives plus 1e-6 / 2^-7 of rounding: 1e-2."""
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 90, 64, 2, 16, seed=12)
    got = run_bwd(p)
    q = dev(p)
    r = torch.Generator().manual_seed(5)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="dbias",
                 h0="dh0")
    way = {k: torch.randn(q[k].shape, generator=r).cuda() * (0.05 if k == "A" else 1.0)
           for k in names}

    def loss(s):
        v = {k: q[k] + s * way[k] for k in names}
        y, ht = gdn.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"],
                                   dt_bias=v["dt_bias"], dt_softplus=True,
                                   initial_state=v["h0"])
        return float((y.double() * q["dy"].double()).sum() +
                     (ht.double() * q["dht"].double()).sum())

    for k in names:  # one input at a time, so that none hides behind another
        keep, way_all = {}, dict(way)
        for j in names:
            if j != k:
                keep[j], way[j] = way[j], torch.zeros_like(way[j])
        e = 2.0 ** -7
        num = (loss(e) - loss(-e)) / (2 * e)
        want = float((got[names[k]].double() * way[k].double()).sum())
        size = float((got[names[k]].double().norm() * way[k].double().norm()))
        assert abs(num - want) <= 1e-2 * max(abs(want), size / 30), (k, num, want)
        way.update(way_all)


def test_same_bits_again_on_another_stream_and_strided():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(2, 200, 65, 1, 16, "bf16", seed=14)
    first = run_bwd(p)
    q = dev(p)
    xz = torch.zeros(2, 200, 131, dtype=torch.bfloat16, device="cuda")
    xz[..., :65], xz[..., 66:] = q["x"], q["z"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out = gdn.selective_scan_bwd(xz[..., :65], q["dt"], q["A"], q["B"], q["C"], q["dy"],
                                     D=q["D"], z=xz[..., 66:], dt_bias=q["dt_bias"],
                                     dt_softplus=True, initial_state=q["h0"], dht=q["dht"])
    s.synchronize()
    for k, t in zip(NAMES, out):
        assert torch.equal(t, first[k]), k


def test_zero_gradients_in_give_zeros():
    p = make(1, 70, 64, 1, 16, seed=15)
    p["dy"], p["dht"] = torch.zeros_like(p["dy"]), torch.zeros_like(p["dht"])
    for k, t in run_bwd(p).items():
        assert not t.any(), k


def test_no_sequences():
    import gated_deltanet_chunked_02_amd as gdn
    p = make(1, 5, 64, 1, 16, h0=False, seed=16)
    q = dev(p)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.selective_scan_bwd(q["x"], q["dt"], q["A"], q["B"], q["C"], q["dy"], D=q["D"],
                                 dt_bias=q["dt_bias"], cu_seqlens=cu)
    assert not out[2].any() and not out[5].any() and not out[7].any()
