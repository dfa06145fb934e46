"""The example layer, which runs the state-space calls together as a model does."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_layer_decodes_as_it_reads_and_learns():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import selective_layer
    err, losses = selective_layer.main()
    # every activation is rounded to bf16 (2^-8) on both sides, at slightly different values after
    # each of the five stages: 5 x 2^-8
    assert err <= 5 * 2.0 ** -8, err
    assert losses[-1] < losses[0], losses


def test_layer_replays_from_a_graph():
    """A prompt and a token captured once and replayed on changed inputs give the eager calls' bits:
    nothing in them depends on the host after the capture."""
    import gated_deltanet_chunked_02_amd as gdn
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    C, S, T = 320, 16, 600
    A = -torch.arange(1, S + 1).float().repeat(C, 1).cuda()
    D, w = n(C), n(C, 4)
    x, dt, z, dy = (n(1, T, C).bfloat16() for _ in range(4))
    B, Cm = n(1, T, 1, S).bfloat16(), n(1, T, 1, S).bfloat16()
    state = torch.zeros(1, C, S, device="cuda")

    def run():
        u = gdn.causal_conv1d(x, w, activation="silu")
        y, ht = gdn.selective_scan(u, dt, A, B, Cm, D=D, z=z, dt_softplus=True)
        state.copy_(ht)
        last = gdn.selective_state_update(state, u[:, 0], dt[:, 0], A, B[:, 0], Cm[:, 0], D=D,
                                          z=z[:, 0], dt_softplus=True)
        v, mean, rstd = gdn.group_norm(y.view(T, C), 5, activation="silu")
        grads = gdn.selective_scan_bwd(u, dt, A, B, Cm, dy, D=D, z=z, dt_softplus=True)
        dx, dw, _, _ = gdn.causal_conv1d_bwd(x, w, grads[0], activation="silu")
        dn = gdn.group_norm_bwd(dy.view(T, C), y.view(T, C), 5, mean, rstd, activation="silu")
        return [last, v, state, dx, dw, *grads, *dn]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(4):
        x.copy_(n(1, T, C))
        dt.copy_(n(1, T, C))
        graph.replay()
        torch.cuda.synchronize()
        got = [None if t is None else t.clone() for t in held]
        want = run()
        for i, (a, b) in enumerate(zip(got, want)):
            assert (a is None) == (b is None), i
            assert a is None or torch.equal(a, b), i
