"""Linear attention and its gradient on long walks against the fp64 oracle: sequences over several of the
states kept for the gradient (every 512 tokens in bf16, 256 in fp32, half of that with a head's own
decay), whole, in segments of several such spans, and packed with bounds that fall on none.

Tolerances are those of test_gpu_linear and test_gpu_linear_bwd, whose states are remembered for 20 chunks
at most; the slow decays here, 0.01 a token at most, keep one for 16 chunks in bf16 (e^-10), and a head's own
likewise."""
import pytest
import torch

from test_gpu_linear import TOL, TOL_F32, check, make, oracle_fwd, run_fwd
from test_gpu_linear_bwd import check_all, oracle_bwd, run_bwd

pytestmark = pytest.mark.gpu

WALKS = [
    # T, lens, H, D: whole sequences (a head a CU) over three kept states; segments of 1536 tokens, longer
    # than the span between two, dense and packed
    (1100, None, 256, 8), (4400, None, 64, 8), (0, [100, 3000, 1, 1299], 64, 8)]


def slow(T, lens, H, D, dtype, head):
    p = make(1, T, H, H // 4, D, D, dtype, head, True, lens, seed=H + T)
    g = torch.rand(p["g"].shape, generator=torch.Generator().manual_seed(T))
    p["g"] = -0.01 * (0.5 + 0.5 * g)
    return p


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens,H,D", WALKS)
def test_long_walks_match_oracle(T, lens, H, D, dtype, head):
    p = slow(T, lens, H, D, dtype, head)
    o_ref, ht_ref = oracle_fwd(p)
    o, ht = run_fwd(p)
    check("o", o, o_ref, TOL[dtype])
    check("ht", ht, ht_ref, TOL_F32)
    check_all(p, run_bwd(p), oracle_bwd(p), dtype)
