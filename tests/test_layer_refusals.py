"""What the state-space layer's calls refuse, on the host (no GPU needed): the C ABI's checks before
any launch and the binding's before any pointer reaches it."""
import ctypes

import pytest
import torch

import gated_deltanet_chunked_02_amd as gdn
from gated_deltanet_chunked_02_amd.ssm import _rows

A = 0x10000  # an aligned address that no refused call reads


def scan_desc(**kw):
    base = dict(B=2, T=100, N=2, channels=128, groups=2, dstate=16, dtype=1, dt_softplus=1,
                state_lines=4)
    base.update(kw)
    return gdn.GdnScanDesc(**base)


def conv_desc(**kw):
    base = dict(B=2, T=100, N=2, channels=64, width=4, dtype=1, activation=1, state_lines=0)
    base.update(kw)
    return gdn.GdnConvDesc(**base)


def norm_desc(**kw):
    base = dict(samples=2, positions=1000, channels=64, groups=4, dtype=1, activation=1, eps=1e-5)
    base.update(kw)
    return gdn.GdnNormDesc(**base)


def size(name, d, *more):
    st = ctypes.c_int(-1)
    n = getattr(gdn.load(), name)(ctypes.byref(d), *more, ctypes.byref(st))
    return st.value, n


SCAN_BAD = [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(N=-1), 1), (dict(channels=0), 1), (dict(groups=0), 1),
    (dict(channels=127), 1), (dict(dstate=0), 1), (dict(dtype=2), 1), (dict(dt_softplus=2), 1),
    (dict(N=3), 1), (dict(x_stride=127), 1), (dict(dt_stride=-1), 1), (dict(z_stride=64), 1),
    (dict(b_stride=31), 1), (dict(c_stride=31), 1), (dict(dstate=257), 2),
    (dict(B=1 << 16, T=1 << 16, N=0), 2), (dict(channels=1 << 21), 2),
    # a row so long that a tile of them passes 2 GiB; more B and C values than a launch has threads
    (dict(x_stride=1 << 24), 2), (dict(B=1 << 15, N=0, T=1 << 12, groups=8, dstate=16), 2),
]


@pytest.mark.parametrize("kw,status", SCAN_BAD)
def test_scan_descriptors(kw, status):
    for name in ("gdn_selective_scan_workspace_size", "gdn_selective_scan_bwd_workspace_size"):
        assert size(name, scan_desc(**kw)) == (status, 0)
    d = scan_desc(**kw)
    assert gdn.gdn_selective_scan_fwd(d, *[A] * 9, None, A, A, 0) == status
    assert gdn.gdn_selective_scan_bwd(d, *[A] * 9, None, *[A] * 11, 0) == status


def test_scan_pointers_and_workspace():
    need = size("gdn_selective_scan_workspace_size", scan_desc())[1]
    assert need > 0
    d = scan_desc(workspace=A, workspace_bytes=need)
    good = [A] * 9 + [None, A, A]
    for i in (0, 1, 2, 3, 4, 10):  # x, dt, A, B, C, y are required
        assert gdn.gdn_selective_scan_fwd(d, *good[:i], None, *good[i + 1:], 0) == 1, i
    for i, off in ((0, 1), (2, 2), (5, 2), (7, 1), (8, 1), (11, 2)):  # misaligned
        assert gdn.gdn_selective_scan_fwd(d, *good[:i], A + off, *good[i + 1:], 0) == 1, i
    for kw in (dict(workspace=None, workspace_bytes=need),
               dict(workspace=A, workspace_bytes=need - 1),
               dict(workspace=A + 16, workspace_bytes=need)):
        assert gdn.gdn_selective_scan_fwd(scan_desc(**kw), *good, 0) == 3
    need = size("gdn_selective_scan_bwd_workspace_size", scan_desc())[1]
    good = [A] * 9 + [None, A, A] + [A] * 9
    d = scan_desc(workspace=A, workspace_bytes=need)
    for i in (0, 1, 2, 3, 4, 10, 12, 13, 14, 15, 16, 18):  # z needs dz
        assert gdn.gdn_selective_scan_bwd(d, *good[:i], None, *good[i + 1:], 0) == 1, i
    d = scan_desc(workspace=A, workspace_bytes=need - 1)
    assert gdn.gdn_selective_scan_bwd(d, *good, 0) == 3


def test_scan_workspace_covers_dense_and_packed():
    """A descriptor of one sequence may be used either way: the query gives the larger need."""
    one = scan_desc(B=1, N=1, T=4000, channels=64, groups=1)
    dense = size("gdn_selective_scan_workspace_size", one)
    two = scan_desc(B=1, N=2, T=4000, channels=64, groups=1)
    assert dense[0] == 0 and 0 < dense[1] <= size("gdn_selective_scan_workspace_size", two)[1]


def test_step_refusals():
    args = [A] * 9 + [None, None, A]
    assert gdn.gdn_selective_state_update(scan_desc(), *args, 0) == 1            # T is not 1
    assert gdn.gdn_selective_state_update(scan_desc(T=1, state_lines=0), *args, 0) == 1
    d = scan_desc(T=1)
    for i in (0, 1, 2, 3, 4, 5, 11):
        assert gdn.gdn_selective_state_update(d, *args[:i], None, *args[i + 1:], 0) == 1, i
    assert gdn.gdn_selective_state_update(d, A + 2, *args[1:], 0) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(channels=0), 1), (dict(dtype=9), 1), (dict(activation=5), 1),
    (dict(N=5), 1), (dict(width=1), 2), (dict(width=5), 2), (dict(channels=12), 2),
    (dict(B=1 << 16, T=1 << 16, N=0), 2)])
def test_conv_gradient_descriptors(kw, status):
    d = conv_desc(**kw)
    if kw != dict(N=5):  # which reads as a packed batch in the query
        assert size("gdn_causal_conv1d_bwd_workspace_size", d) == (status, 0)
    assert gdn.gdn_causal_conv1d_bwd(d, *[A] * 4, None, *[A] * 7, 1 << 30, 0) == status


def test_conv_gradient_pointers_and_workspace():
    d = conv_desc()
    need = size("gdn_causal_conv1d_bwd_workspace_size", d)[1]
    good = [A] * 4 + [None] + [A] * 7
    for i in (0, 1, 5, 7):
        assert gdn.gdn_causal_conv1d_bwd(d, *good[:i], None, *good[i + 1:], need, 0) == 1, i
    for i in (0, 3, 5, 6, 7, 10):
        assert gdn.gdn_causal_conv1d_bwd(d, *good[:i], A + 8, *good[i + 1:], need, 0) == 1, i
    assert gdn.gdn_causal_conv1d_bwd(d, *good, need - 1, 0) == 3
    assert gdn.gdn_causal_conv1d_bwd(d, *good[:11], None, need, 0) == 3


@pytest.mark.parametrize("kw,status", [
    (dict(samples=-1), 1), (dict(positions=-1), 1), (dict(channels=0), 1), (dict(groups=0), 1),
    (dict(groups=5), 1), (dict(dtype=2), 1), (dict(activation=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(samples=1 << 22), 2),
    (dict(samples=1 << 22, positions=1, channels=1032, groups=1), 2)])
def test_norm_descriptors(kw, status):
    d = norm_desc(**kw)
    assert size("gdn_group_norm_workspace_size", d, 1) == (status, 0)
    assert gdn.gdn_group_norm_fwd(d, *[A] * 7, 0) == status
    assert gdn.gdn_group_norm_bwd(d, *[A] * 11, 0) == status


def test_norm_pointers_and_workspace():
    need = size("gdn_group_norm_workspace_size", norm_desc(), 0)[1]
    assert need > 0
    d = norm_desc(workspace=A, workspace_bytes=need)
    good = [A] * 7
    for i in (0, 4):
        assert gdn.gdn_group_norm_fwd(d, *good[:i], None, *good[i + 1:], 0) == 1, i
    for i, off in ((0, 1), (1, 2), (3, 1), (4, 1), (5, 2)):
        assert gdn.gdn_group_norm_fwd(d, *good[:i], A + off, *good[i + 1:], 0) == 1, i
    assert gdn.gdn_group_norm_fwd(norm_desc(), *good, 0) == 3
    good = [A] * 11
    need = size("gdn_group_norm_workspace_size", norm_desc(), 1)[1]
    d = norm_desc(workspace=A, workspace_bytes=need)
    for i in (0, 4, 5, 6, 7, 10):
        assert gdn.gdn_group_norm_bwd(d, *good[:i], None, *good[i + 1:], 0) == 1, i
    assert gdn.gdn_group_norm_bwd(norm_desc(workspace=A, workspace_bytes=need - 1), *good, 0) == 3
    # a token's rows need none forward, however many
    assert size("gdn_group_norm_workspace_size", norm_desc(samples=1 << 24, positions=1), 0) == (0, 0)
    assert size("gdn_group_norm_workspace_size", norm_desc(positions=1), 0) == (0, 0)


def scan_tensors():
    r = torch.randn
    return dict(x=r(2, 5, 8), dt=r(2, 5, 8), A=r(8, 4), B=r(2, 5, 2, 4), C=r(2, 5, 2, 4))


@pytest.mark.parametrize("change,error", [
    (dict(x=torch.zeros(2, 5)), ValueError),
    (dict(x=torch.zeros(2, 5, 8, dtype=torch.float16)), TypeError),
    (dict(dt=torch.zeros(2, 5, 7)), ValueError),
    (dict(dt=torch.zeros(2, 5, 8, dtype=torch.bfloat16)), TypeError),
    (dict(A=torch.zeros(7, 4)), ValueError),
    (dict(A=torch.zeros(8, 4, dtype=torch.float64)), TypeError),
    (dict(B=torch.zeros(2, 5, 3, 4), C=torch.zeros(2, 5, 3, 4)), ValueError),
    (dict(C=torch.zeros(2, 5, 2, 5)), ValueError),
    (dict(C=torch.zeros(2, 5, 1, 4)), ValueError),
    (dict(D=torch.zeros(4)), ValueError),
    (dict(z=torch.zeros(2, 5, 8, dtype=torch.bfloat16)), TypeError),
    (dict(dt_bias=torch.zeros(8, dtype=torch.bfloat16)), TypeError),
    (dict(initial_state=torch.zeros(3, 8, 4)), ValueError),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError),  # B is 2
    (dict(cu_seqlens=torch.zeros(3)), TypeError),
    (dict(), ValueError),  # host tensors
])
def test_binding_checks_the_scan(change, error):
    kw = {**scan_tensors(), **change}
    with pytest.raises(error):
        gdn.selective_scan(**kw)
    with pytest.raises(error):
        gdn.selective_scan_bwd(dy=torch.zeros(2, 5, 8), **kw)


def test_binding_checks_the_gradients_and_the_step():
    t = scan_tensors()
    with pytest.raises(ValueError):
        gdn.selective_scan_bwd(dy=torch.zeros(2, 5, 7), **t)
    with pytest.raises(TypeError):
        gdn.selective_scan_bwd(dy=torch.zeros(2, 5, 8, dtype=torch.bfloat16), **t)
    with pytest.raises(ValueError):
        gdn.selective_scan_bwd(dy=torch.zeros(2, 5, 8), dht=torch.zeros(2, 8, 5), **t)
    one = {k: (v if k == "A" else v[:, 0]) for k, v in t.items()}
    for state in (torch.zeros(2, 8, 5), torch.zeros(1, 8, 4), torch.zeros(0, 8, 4)):
        with pytest.raises(ValueError):
            gdn.selective_state_update(state, **one)
    with pytest.raises(TypeError):
        gdn.selective_state_update(torch.zeros(2, 4, 8).transpose(1, 2), **one)
    with pytest.raises(ValueError):
        gdn.selective_state_update(torch.zeros(2, 8, 4), cache_indices=torch.zeros(3).int(), **one)
    with pytest.raises(TypeError):
        gdn.selective_state_update(torch.zeros(2, 8, 4), cache_indices=torch.zeros(2), **one)


def test_binding_checks_the_convolution_and_the_norm():
    x, w = torch.zeros(1, 5, 8), torch.zeros(8, 4)
    with pytest.raises((TypeError, ValueError)):
        gdn.causal_conv1d_bwd(x, w, torch.zeros(1, 5, 8))  # host tensors
    with pytest.raises(ValueError):
        gdn.causal_conv1d_bwd(x, torch.zeros(7, 4), x)
    n = torch.zeros(3, 8)
    for bad in (dict(num_groups=3), dict(num_groups=0), dict(num_groups=2, weight=torch.zeros(7)),
                dict(num_groups=2, gate=torch.zeros(3, 4)), dict(num_groups=2, eps=-1.0),
                dict(num_groups=2, activation="gelu"), dict(num_groups=2)):
        with pytest.raises(ValueError):
            gdn.group_norm(n, **bad)
    with pytest.raises(TypeError):
        gdn.group_norm(n.half(), 2)
    with pytest.raises(ValueError):
        gdn.group_norm_bwd(n, n, 2, torch.zeros(3, 4), torch.zeros(3, 2))


def test_rows_that_can_be_read_in_place():
    t = torch.zeros(4, 6, 20)
    assert _rows(t, 2) == (t, 0)
    v = t[..., 3:10]
    assert _rows(v, 2)[0] is v and _rows(v, 2)[1] == 20
    g = v[..., :6].unflatten(-1, (2, 3))
    assert _rows(g, 2)[0] is g and _rows(g, 2)[1] == 20
    one = t[:1, :, 3:10]
    assert _rows(one, 2) == (one, 20)
    for other in (t[:, ::2], t.transpose(0, 1), t[:, :1].expand(4, 6, 20), t[..., ::2],
                  t[:, :3, :5]):
        got, stride = _rows(other, 2)
        if not (got is other):
            assert got.is_contiguous() and stride == 0 and torch.equal(got, other)
    # every second token of a single sequence is evenly spaced
    assert _rows(t[:1, ::2], 2)[1] == 40
