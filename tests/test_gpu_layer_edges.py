"""Edges of the norm, the convolution's gradient and the single-token scan on the GPU."""
import pytest
import torch

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
