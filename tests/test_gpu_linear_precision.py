"""How near linear attention's results are to the fp64 oracle's, beyond a tolerance for roundings on the
way: bf16 results are fp32 sums rounded once, and fp32 results of a bf16 call are fp32 sums.

bf16 tensors are compared with the oracle's values rounded to bf16.  A value off by d before its
rounding comes out on the other side of a half step with probability d / step and is then a step away, so
the mean square of the difference is at most sum |d| step <= |d|_2 |step|_2, where a step is at most 2^-7
of its value: the relative L2 difference is at most sqrt(D 2^-7) + D for values off by D before the
rounding, D the tolerance of the fp32 results (test_gpu_linear, test_gpu_linear_bwd).  A single rounding of
an operand to bf16 on the way, of 2^-9 at most a value and 1e-3 in the mean, gives sqrt(1e-3 2^-7) = 2.8e-3.

The final state of one chunk is a sum of at most 64 products and a start state: a rounding (2^-24) for
each addition on a random walk, 18 x 2^-24 at most as in test_gpu_linear.  Two bf16 terms for an operand would
leave 2^-18 and more of every product."""
import pytest
import torch

from test_gpu_linear import TOL_F32, check, host, make, oracle_fwd, run_fwd
from test_gpu_linear_bwd import TOL_F32 as TOL_GRAD, oracle_bwd, run_bwd

pytestmark = pytest.mark.gpu


def once(tol):
    return (tol * 2.0 ** -7) ** 0.5 + tol


def check_rounded(name, got, ref, tol):
    check(name, got, host(torch.from_numpy(ref).float().bfloat16()), once(tol))


CASES = [
    # B, T, H, Hg, Dk, Dv, head, h0: o from the state alone, from scores alone, from both, in segments and
    # whole, from long memories, of every tile size
    (96, 1, 8, 8, 128, 128, False, True),
    (2, 64, 16, 4, 128, 128, False, False),
    (3, 200, 8, 4, 64, 64, False, True),
    (1, 700, 4, 1, 128, 128, True, True),
    (1, 700, 4, 4, 64, 128, False, True),
    (2, 600, 130, 130, 8, 16, True, True),
    (2, 300, 4, 4, 128, 64, True, True),
]


@pytest.mark.parametrize("B,T,H,Hg,Dk,Dv,head,h0", CASES + [(1, 300, 4, 2, 256, 256, True, True)])
def test_outputs_are_rounded_once(B, T, H, Hg, Dk, Dv, head, h0):
    p = make(B, T, H, Hg, Dk, Dv, "bf16", head, h0, seed=B + T)
    o, _ = run_fwd(p)
    check_rounded("o", o, oracle_fwd(p)[0], TOL_F32)


@pytest.mark.parametrize("B,T,H,Hg,Dk,Dv,head,h0", CASES)
def test_gradients_are_rounded_once(B, T, H, Hg, Dk, Dv, head, h0):
    p = make(B, T, H, Hg, Dk, Dv, "bf16", head, h0, seed=B + T)
    got, ref = run_bwd(p), oracle_bwd(p)
    for x in ("dq", "dk", "dv"):
        check_rounded(x, got[x], ref[x], TOL_GRAD)


@pytest.mark.parametrize("T", [1, 17, 64])
def test_state_of_a_chunk_is_an_fp32_sum(T):
    p = make(4, T, 8, 4, 128, 128, "bf16", h0=False, seed=T)
    check("ht", run_fwd(p)[1], oracle_fwd(p)[1], 18 * 2.0 ** -24)
