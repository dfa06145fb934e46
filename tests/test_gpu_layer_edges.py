"""Edges of the norm, the convolution's gradient and the single-token scan on the GPU."""
import pytest
import torch

from test_gpu_layer import test_norm_matches_oracle as norm_matches_oracle

pytestmark = pytest.mark.gpu


def test_statistics_of_no_positions():
    """Zero values have no mean: NaN, as the definition's 0 / 0, and not what the memory held."""
    import gated_deltanet_chunked_02_amd as gdn
    held = torch.full((3 * 4 * 2,), 7.0, device="cuda")  # what the statistics' memory may hold
    del held
    x = torch.zeros(3, 0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = gdn.group_norm(x, 4, weight=w)
    assert y.shape == (3, 0, 64) and mean.isnan().all() and rstd.isnan().all()
    assert mean.shape == rstd.shape == (3, 4)
    dx, dw, _, _ = gdn.group_norm_bwd(x, x, 4, mean, rstd, weight=w)
    assert dx.shape == x.shape and not dw.any()
    y, mean, _ = gdn.group_norm(torch.zeros(0, 5, 64, device="cuda"), 4)
    assert y.shape == (0, 5, 64) and mean.shape == (0, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,groups,silu,gated,affine", [
    ((1, 1000, 512), 1, True, False, True),    # 16 slabs of a group of 512 channels
    ((2, 3000, 520), 1, False, True, True),    # 94
    ((1, 700, 333), 3, True, True, False),     # odd: single values
    ((3, 900, 1024), 4, True, False, True),
    ((1, 33, 4100), 2, True, True, True),      # wide rows, few slabs
])
def test_norm_of_wide_groups(shape, groups, dtype, silu, gated, affine):
    """Groups of so many pieces that these are folded over the slabs first."""
    norm_matches_oracle(shape, groups, dtype, silu, gated, affine)


def test_norm_of_wide_groups_far_from_zero_and_with_one_infinity():
    import gated_deltanet_chunked_02_amd as gdn
    from oracle import norm
    from test_gpu_layer import check, host
    x = torch.randn(2, 900, 512, generator=torch.Generator().manual_seed(2)) + 4096.0
    y, mean, rstd = gdn.group_norm(x.cuda(), 2)
    y_ref, _, rstd_ref = norm.group_norm(host(x), 2)
    # x - mean loses no more than 4096 x 2^-23 x 2 of the deviation
    check("y", y, y_ref, 1e-3)
    check("rstd", rstd, rstd_ref, 1e-3)
    x[0, 17, 300] = float("inf")  # sample 0, group 1
    z = gdn.group_norm(x.cuda(), 2)[0]
    assert z[0, ..., 256:].isnan().any()
    z[0, ..., 256:], y[0, ..., 256:] = 0, 0
    assert torch.equal(z, y)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("S", [1, 5, 16, 40])
def test_one_bad_input_stays_in_its_channel_and_sequence(S, bad):
    """In the last channel of a group, whose workgroup has lanes without a channel."""
    from test_gpu_selective import make, run_fwd
    from test_gpu_selective_bwd import run_bwd
    lens, C, G = [50, 40, 260], 70, 2
    p = make(C=C, G=G, S=S, dtype="f32", lens=lens, seed=S)
    clean = dict(zip(("y", "ht"), run_fwd(p)), **run_bwd(p))
    others = [c for c in range(C) if c != 34]
    for key in ("x", "dt", "z", "dy"):
        q = dict(p, **{key: p[key].clone()})
        q[key][0, 60, 34] = bad  # token 10 of sequence 1
        got = dict(zip(("y", "ht"), run_fwd(q)), **run_bwd(q))
        for k in ("y", "dx", "ddt", "dz"):  # [1, T, C]
            assert torch.equal(got[k][..., others], clean[k][..., others]), (key, k)
            for cut in (slice(0, 50), slice(90, None)):
                assert torch.equal(got[k][:, cut], clean[k][:, cut]), (key, k)
        for k in ("dB", "dC"):  # [1, T, G, S]
            assert torch.equal(got[k][:, :, 1], clean[k][:, :, 1]), (key, k)
            for cut in (slice(0, 50), slice(90, None)):
                assert torch.equal(got[k][:, cut], clean[k][:, cut]), (key, k)
        for k in ("ht", "dh0"):  # [N, C, S]
            assert torch.equal(got[k][:, others], clean[k][:, others]), (key, k)
            assert torch.equal(got[k][[0, 2]], clean[k][[0, 2]]), (key, k)
        for k in ("dA", "dD", "dbias"):
            assert torch.equal(got[k][others], clean[k][others]), (key, k)
        if key != "dy":
            assert not got["y"][0, 60, 34].isfinite()
