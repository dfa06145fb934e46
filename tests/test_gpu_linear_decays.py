"""What linear attention's gradient leaves of decays that leave nothing, against the fp64 oracle (tolerances of
test_gpu_linear_bwd)."""
import pytest
import torch

from test_gpu_linear import make
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
