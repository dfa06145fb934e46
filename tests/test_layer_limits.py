"""Sizes at the limits of the state-space layer's calls, on the host (no GPU needed): what is refused
before any launch, and what must not be.  Calls that pass the descriptor's checks are given no
pointers, so that nothing is launched."""
import pytest

import gated_deltanet_chunked_02_amd as gdn
from test_layer_refusals import A, conv_desc, norm_desc, scan_desc, size


@pytest.mark.parametrize("positions,status", [((1 << 31) - 1, 2), ((1 << 30) + 1, 2), (1 << 30, 0)])
def test_norm_positions(positions, status):
    """A pass over positions steps past the last one by up to 2^19: that must stay below 2^31."""
    d = norm_desc(samples=1, positions=positions, channels=1, groups=1)
    for backward in (0, 1):
        got, need = size("gdn_group_norm_workspace_size", d, backward)
        assert got == status and (need > 0) == (status == 0)
    if status:
        assert gdn.gdn_group_norm_fwd(d, *[A] * 7, 0) == status
        assert gdn.gdn_group_norm_bwd(d, *[A] * 11, 0) == status


def test_rows_far_apart():
    """Token t of a [4, 1024, 4096] tensor, and a prompt of one token there: 8 MB from row to row.
    A prompt of three tokens may be 256 MB a row, not 512."""
    far = dict(B=4, N=4, T=1, channels=4096, groups=1)
    for strides in (dict(x_stride=1 << 22), dict(dt_stride=1 << 22, z_stride=1 << 40)):
        d = scan_desc(**far, **strides)
        assert gdn.gdn_selective_state_update(d, A, None, *[A] * 7, None, None, A, 0) == 1
        for name in ("gdn_selective_scan_workspace_size", "gdn_selective_scan_bwd_workspace_size"):
            assert size(name, d)[0] == 0
    for log, status in ((27, 0), (28, 2)):  # bf16 elements
        d = scan_desc(B=1, N=1, T=3, channels=64, groups=1, x_stride=1 << log)
        for name in ("gdn_selective_scan_workspace_size", "gdn_selective_scan_bwd_workspace_size"):
            assert size(name, d)[0] == status
    # and of any length where 257 rows lie within 2 GiB
    for log, status in ((21, 0), (22, 2)):
        d = scan_desc(B=1, N=1, T=100000, channels=64, groups=1, x_stride=1 << log)
        assert size("gdn_selective_scan_workspace_size", d)[0] == status


@pytest.mark.parametrize("kw,forward,backward", [
    # 16384 x 258 workgroups of 1024 threads for the sums of dA, dD and d(dt_bias)
    (dict(B=1, N=1, T=4, channels=1 << 20, groups=1, dstate=256), 0, 2),
    (dict(B=1, N=1, T=4, channels=1 << 20, groups=1, dstate=240), 0, 0),
    # 2^32 - 2^22 values of B and C, and the channels' 2 x 18 workgroups with them
    (dict(B=1, N=1, T=(1 << 27) - (1 << 17), channels=128, groups=1, dstate=16), 0, 0),
    (dict(B=1, N=1, T=(1 << 27) - 32, channels=128, groups=1, dstate=16), 0, 2),
])
def test_gradient_sums_fit_a_launch(kw, forward, backward):
    d = scan_desc(**kw)
    assert size("gdn_selective_scan_workspace_size", d)[0] == forward
    assert size("gdn_selective_scan_bwd_workspace_size", d)[0] == backward
    if backward:
        d.workspace, d.workspace_bytes = A, 1 << 62
        assert gdn.gdn_selective_scan_bwd(d, *[A] * 9, None, *[A] * 11, 0) == backward


def test_any_number_of_groups():
    """65536 and more blocks of channels, as one channel a group makes of 70000."""
    d = scan_desc(B=2, N=2, T=5, channels=70000, groups=70000, dstate=1)
    for name in ("gdn_selective_scan_workspace_size", "gdn_selective_scan_bwd_workspace_size"):
        assert size(name, d)[0] == 0
    d.T = 1
    assert gdn.gdn_selective_state_update(d, A, None, *[A] * 7, None, None, A, 0) == 1


@pytest.mark.parametrize("channels,status", [(65535 * 1024, 0), (65535 * 1024 + 8, 2), (1 << 27, 2)])
def test_conv_gradient_channels(channels, status):
    """Blocks of 1024 channels are a grid's y axis."""
    d = conv_desc(B=1, N=1, T=1, channels=channels)
    assert size("gdn_causal_conv1d_bwd_workspace_size", d)[0] == status
    if status:
        assert gdn.gdn_causal_conv1d_bwd(d, *[A] * 4, None, *[A] * 7, 1 << 62, 0) == status
