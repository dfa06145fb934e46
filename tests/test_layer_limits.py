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
