"""Linear attention where decays leave nothing, its gradient against the fp64 oracle (tolerances of
test_gpu_linear_bwd), and where states are infinite."""
import pytest
import torch

from test_gpu_linear import make, run_fwd
from test_gpu_linear_bwd import check_all, oracle_bwd, run_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(70, 4), (700, 4), (1100, 256)])
def test_decay_of_nothing_left_has_no_gradient(T, H, dtype):
    """A head whose decay leaves nothing of a state, beside others: its dg is 0."""
    p = make(1, T, H, H, 16, 16, dtype, True, seed=T)
    gone = [0, H // 2, H - 1]
    p["g"][gone] = torch.tensor([-float("inf"), -1e30, -200.0])
    got = run_bwd(p)
    check_all(p, got, oracle_bwd(p), dtype)
    assert not bool(got["dg"][gone].any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [70, 700])
def test_infinite_states_stay_in_their_head_and_sequence(T, dtype):
    p = make(2, T, 4, 2, 64, 40, dtype, seed=T)
    fwd, grads = run_fwd(p), run_bwd(p)
    p["h0"][1, 2, 3, 5] = float("inf")
    p["dht"][1, 2, 3, 5] = -float("inf")
    (o, ht), got = run_fwd(p), run_bwd(p)
    assert not bool(o[1, :, 2].isfinite().all()) and not bool(ht[1, 2].isfinite().all())
    for h in range(4):
        for n in range(2):
            if (n, h) == (1, 2):
                continue
            assert torch.equal(o[n, :, h], fwd[0][n, :, h]) and torch.equal(ht[n, h], fwd[1][n, h])
            for x in ("dv", "dg"):
                assert torch.equal(got[x][n, :, h], grads[x][n, :, h]), x
            assert torch.equal(got["dh0"][n, h], grads["dh0"][n, h])
    for x in ("dq", "dk"):  # of the other q/k head
        assert torch.equal(got[x][:, :, 0], grads[x][:, :, 0]) and torch.equal(got[x][0], grads[x][0])
