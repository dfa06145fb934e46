"""The state-space layer's calls on tensors of more than 2^31 elements: what a call gives near their end
against the same call on that part alone.

Tolerances, relative L2: both sides round a bf16 output once, of fp32 values that agree to 1e-5 (the
scan's chunks differ), so they differ by less than one rounding, 2^-8 + 1e-5; fp32 outputs 1e-5."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, C, S, TAIL = 540672, 4096, 16, 700
BF16_TOL, F32_TOL = 2.0 ** -8 + 1e-5, 1e-5


def randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def close(got, want, tol):
    got, want = got.float(), want.float()
    assert got.shape == want.shape and got.isfinite().all()
    assert float((got - want).norm()) <= tol * float(want.norm())


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def test_scan_and_its_gradient():
    import gated_deltanet_chunked_02_amd as gdn
    x, dt = randn(1, T, C, seed=1), randn(1, T, C, seed=2)
    B, Cm = randn(1, T, 1, S, seed=3), randn(1, T, 1, S, seed=4)
    A = -torch.arange(1, S + 1, device="cuda").float().repeat(C, 1)
    kw = dict(dt_bias=torch.full((C,), -2.0, device="cuda"), dt_softplus=True)
    assert x.numel() > 2 ** 31
    y, ht = gdn.selective_scan(x, dt, A, B, Cm, **kw)
    head = [t[:, :-TAIL] for t in (x, dt, B, Cm)]
    tail = [t[:, -TAIL:].clone() for t in (x, dt, B, Cm)]
    _, h0 = gdn.selective_scan(head[0], head[1], A, *head[2:], **kw)
    y1, ht1 = gdn.selective_scan(*tail[:2], A, *tail[2:], initial_state=h0, **kw)
    close(y[:, -TAIL:], y1, BF16_TOL)
    close(ht, ht1, F32_TOL)
    # h0 above came from a call on most of it: the tail must also follow from a short one before it
    near = [t[:, -4 * TAIL:-TAIL].clone() for t in (x, dt, B, Cm)]
    _, h0 = gdn.selective_scan(near[0], near[1], A, *near[2:], **kw)
    _, ht2 = gdn.selective_scan(*tail[:2], A, *tail[2:], initial_state=h0, **kw)
    close(ht, ht2, F32_TOL)
    del y, y1
    dy = randn(1, T, C, seed=5)
    dx, ddt, _, dB, dC = gdn.selective_scan_bwd(x, dt, A, B, Cm, dy, **kw)[:5]
    want = gdn.selective_scan_bwd(*tail[:2], A, *tail[2:], dy[:, -TAIL:].clone(), initial_state=h0,
                                  **kw)
    for got, ref in ((dx, want[0]), (ddt, want[1]), (dB, want[3]), (dC, want[4])):
        close(got[:, -TAIL:], ref, BF16_TOL)


def test_state_pool():
    import gated_deltanet_chunked_02_amd as gdn
    lines = 2 ** 31 // (C * S) + 7
    pool = torch.zeros(lines, C, S, device="cuda")
    one = [randn(3, C, seed=1), randn(3, C, seed=2)]
    B, Cm = randn(3, 1, S, seed=3), randn(3, 1, S, seed=4)
    A = -torch.arange(1, S + 1, device="cuda").float().repeat(C, 1)
    start = randn(3, C, S, seed=5, dtype=torch.float32)
    at = torch.tensor([lines - 1, 0, lines - 5], device="cuda")
    pool[at] = start
    y = gdn.selective_state_update(pool, *one, A, B, Cm, dt_softplus=True, cache_indices=at)
    y1 = gdn.selective_state_update(start, *one, A, B, Cm, dt_softplus=True)
    assert torch.equal(y, y1) and torch.equal(pool[at], start)
    assert not pool[1:lines - 5].any()


def test_conv_gradient():
    import gated_deltanet_chunked_02_amd as gdn
    x, dy = randn(1, T, C, seed=1), randn(1, T, C, seed=2)
    w = randn(C, 4, seed=3, dtype=torch.float32)
    dx = gdn.causal_conv1d_bwd(x, w, dy, activation="silu")[0]
    part = gdn.causal_conv1d_bwd(x[:, -TAIL:].clone(), w, dy[:, -TAIL:].clone(),
                                 initial_state=x[:, -TAIL - 3:-TAIL].clone(), activation="silu")[0]
    assert torch.equal(dx[:, -TAIL:], part)


def test_norm_rows():
    import gated_deltanet_chunked_02_amd as gdn
    x, gate = randn(T, C, seed=1), randn(T, C, seed=2)
    w = randn(C, seed=3, dtype=torch.float32)
    y, mean, rstd = gdn.group_norm(x, 32, w, activation="silu", gate=gate)
    a = gdn.group_norm(x[-TAIL:].clone(), 32, w, activation="silu", gate=gate[-TAIL:].clone())
    for got, want in zip((y, mean, rstd), a):
        assert torch.equal(got[-TAIL:], want)
    dx, _, _, dgate = gdn.group_norm_bwd(y, x, 32, mean, rstd, w, activation="silu", gate=gate)
    b = gdn.group_norm_bwd(a[0], x[-TAIL:].clone(), 32, a[1], a[2], w, activation="silu",
                           gate=gate[-TAIL:].clone())
    assert torch.equal(dx[-TAIL:], b[0]) and torch.equal(dgate[-TAIL:], b[3])


def test_norm_maps():
    """Two maps, the second beginning near 2^31 elements: as that map alone (its sums are split
    otherwise, so to rounding)."""
    import gated_deltanet_chunked_02_amd as gdn
    x, dy = randn(2, T // 2 + 3, C, seed=1), randn(2, T // 2 + 3, C, seed=2)
    w = randn(C, seed=3, dtype=torch.float32)
    y, mean, rstd = gdn.group_norm(x, 32, w, activation="silu")
    grads = gdn.group_norm_bwd(dy, x, 32, mean, rstd, w, activation="silu")
    y1, mean1, rstd1 = gdn.group_norm(x[1:].clone(), 32, w, activation="silu")
    close(y[1:, -TAIL:], y1[:, -TAIL:], BF16_TOL)
    close(rstd[1:], rstd1, F32_TOL)
    assert float((mean[1:] - mean1).abs().max()) <= 1e-6  # of values of deviation 1
    dx1 = gdn.group_norm_bwd(dy[1:].clone(), x[1:].clone(), 32, mean1, rstd1, w,
                             activation="silu")[0]
    close(grads[0][1:, -TAIL:], dx1[:, -TAIL:], BF16_TOL)
