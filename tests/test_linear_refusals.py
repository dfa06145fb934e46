"""What linear attention and the block norm refuse, and what their bindings hand to the library, on the
host (no GPU needed): the C ABI's checks before any launch, sizes at the limits, the binding's checks
before any pointer reaches the library, and the device its calls are made on.  Calls of a descriptor
that passes are given a pointer, a workspace or a size that does not, so that nothing is launched."""
import pytest
import torch

import gated_deltanet_chunked_02_amd as gdn
from test_layer_binding import BIG, Recorder, meta
from test_layer_refusals import A, size

BF16, F32 = torch.bfloat16, torch.float32
SIZES = ("gdn_linear_attn_workspace_size", "gdn_linear_attn_bwd_workspace_size")


def linear_desc(**kw):
    base = dict(B=2, T=4000, N=2, H=8, Hg=4, Dk=64, Dv=64, dtype=1, head_decay=0, state_lines=4,
                scale=0.125)
    base.update(kw)
    return gdn.GdnLinearDesc(**base)


def block_desc(**kw):
    base = dict(rows=40, channels=64, dtype=1, residual_dtype=1, post_norm=1, activation=1,
                eps=1e-5, residual_scale=1.0)
    base.update(kw)
    return gdn.GdnBlockNormDesc(**base)


FWD = [A] * 5 + [None] + [A] * 2      # q k v g h0 cu o ht
BWD = [A] * 5 + [None] + [A] * 7      # q k v g h0 cu do dht dq dk dv dg dh0
STEP = [A] * 5 + [None, None, A]      # state q k v g read write o


def put(args, i, value):
    return args[:i] + [value] + args[i + 1:]


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(N=-1), 1), (dict(H=0), 1), (dict(Hg=0), 1),
    (dict(H=6), 1), (dict(Dk=0), 1), (dict(Dv=-8), 1), (dict(dtype=2), 1),
    (dict(head_decay=2), 1), (dict(N=3), 1), (dict(q_stride=255), 1), (dict(q_stride=257), 1),
    (dict(k_stride=-256), 1), (dict(v_stride=508), 1), (dict(Dk=60), 2), (dict(Dv=68), 2),
    (dict(Dk=264), 2), (dict(Dv=264), 2), (dict(v_stride=1 << 23), 2),
    (dict(B=1 << 15, N=0, T=1 << 16), 2), (dict(B=(1 << 16) + 1, N=0, T=1), 2),
    (dict(H=1 << 17, Hg=1), 2),
    # more workgroups than a launch may have
    (dict(B=1 << 16, N=0, T=1, H=256, Hg=256), 2),
])
def test_linear_descriptors(kw, status):
    for name in SIZES:
        assert size(name, linear_desc(**kw)) == (status, 0)
    if kw != dict(N=3):  # which reads as a packed batch in the queries
        d = linear_desc(workspace=A, workspace_bytes=1 << 62, **kw)
        assert gdn.gdn_linear_attn_fwd(d, *FWD, 0) == status
        assert gdn.gdn_linear_attn_bwd(d, *BWD, 0) == status


def test_linear_gradient_heads():
    """Heads of more than 128 have no gradient."""
    for kw in (dict(Dk=136), dict(Dv=256)):
        d = linear_desc(**kw)
        assert size(SIZES[0], d)[0] == 0 and size(SIZES[1], d) == (2, 0)
        assert gdn.gdn_linear_attn_bwd(d, *BWD, 0) == 2


def test_linear_pointers_and_workspace():
    need = size(SIZES[0], linear_desc())[1]
    assert need > 0
    d = linear_desc(workspace=A, workspace_bytes=need)
    for i in (0, 1, 2, 3, 6):
        assert gdn.gdn_linear_attn_fwd(d, *put(FWD, i, None), 0) == 1, i
    for i, off in ((0, 8), (1, 4), (2, 2), (3, 2), (4, 8), (6, 8), (7, 4)):
        assert gdn.gdn_linear_attn_fwd(d, *put(FWD, i, A + off), 0) == 1, i
    assert gdn.gdn_linear_attn_fwd(linear_desc(B=1, N=1), *put(FWD, 5, A + 2), 0) == 1
    for kw in (dict(workspace=None, workspace_bytes=need), dict(workspace=A, workspace_bytes=need - 1),
               dict(workspace=A + 16, workspace_bytes=need)):
        assert gdn.gdn_linear_attn_fwd(linear_desc(**kw), *FWD, 0) == 3
    need = size(SIZES[1], linear_desc())[1]
    d = linear_desc(workspace=A, workspace_bytes=need)
    for i in (0, 1, 2, 3, 6, 8, 9, 10):
        assert gdn.gdn_linear_attn_bwd(d, *put(BWD, i, None), 0) == 1, i
    for i, off in ((0, 8), (4, 4), (6, 2), (7, 8), (8, 8), (9, 2), (10, 4), (11, 2), (12, 8)):
        assert gdn.gdn_linear_attn_bwd(d, *put(BWD, i, A + off), 0) == 1, i
    for kw in (dict(workspace=None, workspace_bytes=need), dict(workspace=A, workspace_bytes=need - 1),
               dict(workspace=A + 16, workspace_bytes=need)):
        assert gdn.gdn_linear_attn_bwd(linear_desc(**kw), *BWD, 0) == 3


def test_linear_workspace():
    """Short sequences take none forward; a packed batch of one no more than the query of one says."""
    assert size(SIZES[0], linear_desc(T=100)) == (0, 0)
    assert size(SIZES[0], linear_desc(T=0)) == (0, 0)
    one = size(SIZES[0], linear_desc(B=1, N=1))
    two = size(SIZES[0], linear_desc(B=1, N=2))
    assert one[0] == two[0] == 0 and 0 < one[1] <= two[1]
    # a gradient keeps a state every 512 bf16 tokens, 256 fp32 ones
    plain = dict(B=8, N=8, T=2048, H=32, Hg=32, Dk=128, Dv=128)
    states = 8 * 4 * 32 * 128 * 128 * 4
    # (half of that where a head's own decay is wanted), and a number for each token and head
    numbers = 8 * 2048 * 32 * 8
    assert size(SIZES[1], linear_desc(**plain)) == (0, states + numbers)
    assert size(SIZES[1], linear_desc(**{**plain, "dtype": 0})) == (0, 2 * states + numbers)
    sums = 8 * 32 * 8  # of each sequence's dg
    assert size(SIZES[1], linear_desc(**{**plain, "head_decay": 1})) == (0, 2 * states + numbers + sums)


def test_linear_step_refusals():
    assert gdn.gdn_linear_state_update(linear_desc(), *STEP, 0) == 1  # T is not 1
    assert gdn.gdn_linear_state_update(linear_desc(T=1, state_lines=0), *STEP, 0) == 1
    d = linear_desc(T=1)
    for i in (0, 1, 2, 3, 4, 7):
        assert gdn.gdn_linear_state_update(d, *put(STEP, i, None), 0) == 1, i
    for i, off in ((0, 8), (1, 8), (2, 4), (3, 2), (4, 2), (5, 2), (6, 1), (7, 8)):
        assert gdn.gdn_linear_state_update(d, *put(STEP, i, A + off), 0) == 1, i
    d = linear_desc(B=1 << 16, N=0, T=1, H=256, Dv=64)
    assert gdn.gdn_linear_state_update(d, *STEP, 0) == 2


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(channels=0), 1), (dict(dtype=3), 1), (dict(residual_dtype=-1), 1),
    (dict(post_norm=2), 1), (dict(activation=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(h_stride=63), 1), (dict(gate_stride=-64), 1),
    (dict(dtype=0), 2), (dict(rows=(1 << 30) + 1), 2), (dict(channels=(1 << 20) + 1), 2),
    (dict(h_stride=(1 << 32) + 1), 2), (dict(gate_stride=(1 << 32) + 1), 2)])
def test_block_descriptors(kw, status):
    d = block_desc(**kw)
    if "dtype" in kw and status == 2:
        assert d.dtype == 0 and d.residual_dtype == 1  # fp32 blocks beside a bf16 stream
    assert size("gdn_block_norm_bwd_workspace_size", d) == (status, 0)
    assert gdn.gdn_block_norm_fwd(d, *[A] * 10, 0) == status
    assert gdn.gdn_block_norm_bwd(d, *[A] * 16, 0) == status


def test_block_pointers_and_workspace():
    d = block_desc()
    good = [A] * 10  # x h gate post_weight scale weight x_out y post_rstd rstd
    for i in (0, 1, 6):
        assert gdn.gdn_block_norm_fwd(d, *put(good, i, None), 0) == 1, i
    for i, off in ((0, 1), (1, 1), (2, 1), (3, 2), (4, 2), (5, 1), (6, 1), (7, 1), (8, 2), (9, 2)):
        assert gdn.gdn_block_norm_fwd(d, *put(good, i, A + off), 0) == 1, i
    assert gdn.gdn_block_norm_fwd(block_desc(post_norm=0), *good, 0) == 1  # post_weight without it
    assert gdn.gdn_block_norm_fwd(d, A, *[None] * 5, A, None, None, None, 0) == 1  # nothing to make
    need = size("gdn_block_norm_bwd_workspace_size", d)[1]
    assert need > 0
    d = block_desc(workspace=A, workspace_bytes=need)
    # x h gate post_weight scale weight post_rstd rstd dx_out dy dx dh dgate dpost dscale dweight
    good = [A] * 16
    for i in (0, 1, 6, 7, 10, 11, 12):
        assert gdn.gdn_block_norm_bwd(d, *put(good, i, None), 0) == 1, i
    assert gdn.gdn_block_norm_bwd(d, *put(put(good, 8, None), 9, None), 0) == 1
    for i, off in enumerate([1] * 3 + [2] * 5 + [1] * 5 + [2] * 3):
        assert gdn.gdn_block_norm_bwd(d, *put(good, i, A + off), 0) == 1, i
    for kw in (dict(workspace=None, workspace_bytes=need), dict(workspace=A, workspace_bytes=need - 1),
               dict(workspace=A + 16, workspace_bytes=need)):
        assert gdn.gdn_block_norm_bwd(block_desc(**kw), *good, 0) == 3


def tensors(B=2, T=5, H=4, Hg=2, Dk=8, Dv=16, dtype=F32, new=torch.zeros):
    t = dict(q=(B, T, Hg, Dk), k=(B, T, Hg, Dk), v=(B, T, H, Dv))
    return {**{n: new(*s, dtype=dtype) for n, s in t.items()}, "g": new(B, T, H, dtype=F32)}


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros(2, 5, 2)), ValueError),
    (dict(q=None), TypeError),
    (dict(q=torch.zeros(2, 5, 2, 8, dtype=torch.float16)), TypeError),
    (dict(k=torch.zeros(2, 5, 4, 8)), ValueError),
    (dict(k=torch.zeros(2, 5, 2, 8, dtype=BF16)), TypeError),
    (dict(v=torch.zeros(2, 4, 4, 16)), ValueError),
    (dict(v=torch.zeros(2, 5, 3, 16)), ValueError),
    (dict(v=torch.zeros(2, 5, 0, 16)), ValueError),
    (dict(v=torch.zeros(2, 5, 4, 16, dtype=BF16)), TypeError),
    (dict(g=torch.zeros(2, 5, 2)), ValueError),
    (dict(g=torch.zeros(2)), ValueError),
    (dict(g=torch.zeros(2, 5, 4, dtype=BF16)), TypeError),
    (dict(initial_state=torch.zeros(2, 4, 16, 8)), ValueError),
    (dict(initial_state=torch.zeros(2, 4, 8, 16, dtype=BF16)), TypeError),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError),  # B is 2
    (dict(cu_seqlens=torch.zeros(3)), TypeError),
    (dict(), ValueError),  # host tensors
])
def test_binding_checks_linear_attention(change, error):
    kw = {**tensors(), **change}
    with pytest.raises(error):
        gdn.linear_attention(**kw)
    with pytest.raises(error):
        gdn.linear_attention_bwd(do=torch.zeros(2, 5, 4, 16), **kw)


def test_binding_checks_the_gradient_and_the_step():
    t = tensors()
    for do, error in ((torch.zeros(2, 5, 4, 8), ValueError), (None, TypeError),
                      (torch.zeros(2, 5, 4, 16, dtype=BF16), TypeError)):
        with pytest.raises(error):
            gdn.linear_attention_bwd(do=do, **t)
    with pytest.raises(ValueError):
        gdn.linear_attention_bwd(do=t["v"], dht=torch.zeros(2, 4, 16, 8), **t)
    one = {n: x[:, 0] for n, x in t.items()}
    for state in (torch.zeros(2, 4, 16, 8), torch.zeros(1, 4, 8, 16), torch.zeros(0, 4, 8, 16)):
        with pytest.raises(ValueError):
            gdn.linear_state_update(state, **one)
    for state in (torch.zeros(2, 4, 16, 8).transpose(2, 3), torch.zeros(2, 4, 8, 16, dtype=BF16),
                  torch.zeros(1025)[1:].view(2, 4, 8, 16)):
        with pytest.raises(TypeError):
            gdn.linear_state_update(state, **one)
    good = torch.zeros(2, 4, 8, 16)
    with pytest.raises(ValueError):
        gdn.linear_state_update(good, cache_indices=torch.zeros(3).int(), **one)
    with pytest.raises(TypeError):
        gdn.linear_state_update(good, out_indices=torch.zeros(2), **one)
    with pytest.raises(ValueError):
        gdn.linear_state_update(good, **one)  # host tensors


X = torch.zeros(3, 8)


@pytest.mark.parametrize("args,kw,error", [
    ((None,), dict(), TypeError), ((X.half(),), dict(), TypeError),
    ((torch.zeros(8),), dict(), ValueError), ((torch.zeros(3, 0),), dict(), ValueError),
    ((X,), dict(pre_norm=False), ValueError), ((X,), dict(gate=X), ValueError),
    ((X,), dict(post_norm=True), ValueError), ((X,), dict(scale=torch.zeros(8)), ValueError),
    ((X, torch.zeros(3, 7)), dict(), ValueError), ((X, X.half()), dict(), TypeError),
    ((X.bfloat16(), X), dict(), TypeError), ((X, X), dict(dtype=BF16), TypeError),
    ((X, X), dict(gate=X.bfloat16()), TypeError), ((X, X), dict(gate=X[:2]), ValueError),
    ((X, X), dict(weight=torch.zeros(7)), ValueError),
    ((X, X), dict(weight=torch.zeros(8).bfloat16()), TypeError),
    ((X, X), dict(weight=torch.zeros(8), pre_norm=False), ValueError),
    ((X, X), dict(post_weight=torch.zeros(8)), ValueError),
    ((X, X), dict(activation="gelu"), ValueError), ((X, X), dict(eps=-1.0), ValueError),
    ((torch.zeros(8, 3).t(), X), dict(inplace=True), ValueError),
    ((X, X), dict(), ValueError),  # host tensors
])
def test_binding_checks_the_block_norm(args, kw, error):
    with pytest.raises(error):
        gdn.block_norm(*args, **kw)


@pytest.mark.parametrize("change,error", [
    (dict(dy=None, dx=None), TypeError), (dict(dy=torch.zeros(3, 7)), ValueError),
    (dict(dx=X.bfloat16()), TypeError), (dict(rstd=None), TypeError),
    (dict(rstd=torch.zeros(4)), ValueError), (dict(post_norm=True), TypeError),
    (dict(dy=None, weight=torch.zeros(8)), ValueError),
    (dict(), ValueError),  # host tensors
])
def test_binding_checks_the_block_norms_gradient(change, error):
    kw = {**dict(dy=X, dx=X, x=X, h=X, rstd=torch.zeros(3)), **change}
    with pytest.raises(error):
        gdn.block_norm_bwd(**kw)


@pytest.fixture
def recorder(monkeypatch):
    import contextlib
    rec = Recorder(gdn.load())

    @contextlib.contextmanager
    def device(d):
        before, rec.device = rec.device, d
        yield
        rec.device = before

    for module in (gdn, gdn.ssm, gdn.linear, gdn.block):
        monkeypatch.setattr(module, "load", lambda: rec)
    for module in (gdn, gdn.ssm):
        monkeypatch.setattr(module, "_check_devices", lambda *a: None)
    monkeypatch.setattr(gdn, "_raw", (lambda: 0, lambda index: 0))
    monkeypatch.setattr(torch.cuda, "device", device)
    return rec


def linear_args(**kw):
    return {**tensors(new=meta, **kw)}


def step_args(B, lines):
    t = {n: x[:, 0] for n, x in tensors(B=B, new=meta).items()}
    return dict(state=meta(lines, 4, 8, 16), **t)


@pytest.mark.parametrize("call", [
    lambda: gdn.linear_attention(**linear_args(T=BIG, B=1)),
    lambda: gdn.linear_attention(**linear_args(T=1, B=BIG)),
    lambda: gdn.linear_attention(**linear_args(B=1, T=1, Dv=2 ** 32 + 64)),
    lambda: gdn.linear_attention(**linear_args(B=1, T=1, H=2 ** 32 + 4)),
    lambda: gdn.linear_attention(**linear_args(B=1), cu_seqlens=meta(BIG, dtype=torch.int32)),
    lambda: gdn.linear_attention_bwd(**linear_args(B=1, T=BIG), do=meta(1, BIG, 4, 16)),
    lambda: gdn.linear_state_update(**step_args(BIG, BIG)),
    lambda: gdn.linear_state_update(**step_args(2, BIG)),
    lambda: gdn.block_norm(meta(BIG, 8), meta(BIG, 8)),
    lambda: gdn.block_norm(meta(2 ** 16, 2 ** 16, 8)),
    lambda: gdn.block_norm(meta(1, BIG)),
    lambda: gdn.block_norm_bwd(meta(BIG, 8), None, meta(BIG, 8), meta(BIG, 8), rstd=meta(BIG)),
])
def test_sizes_past_32_bits_are_refused(recorder, call):
    with pytest.raises(gdn.GdnError) as e:
        call()
    assert e.value.status == 2 and not recorder.calls


@pytest.mark.parametrize("name,call", [
    ("gdn_linear_attn_fwd", lambda: gdn.linear_attention(**linear_args())),
    ("gdn_linear_attn_bwd", lambda: gdn.linear_attention_bwd(**linear_args(), do=meta(2, 5, 4, 16))),
    ("gdn_linear_state_update", lambda: gdn.linear_state_update(**step_args(2, 3))),
    ("gdn_block_norm_fwd", lambda: gdn.block_norm(meta(3, 8), meta(3, 8))),
    ("gdn_block_norm_bwd", lambda: gdn.block_norm_bwd(meta(3, 8), None, meta(3, 8), meta(3, 8),
                                                      rstd=meta(3))),
])
def test_launches_with_the_tensors_device_current(recorder, name, call):
    """Device 0 is current; the tensors are on another one, whose default stream is 0 as well."""
    call()
    assert [(c[0], c[3]) for c in recorder.calls] == [(name, torch.device("meta"))]
    assert recorder.device == 0


@pytest.mark.parametrize("dtype,width", [(F32, 16), (BF16, 24)])
def test_slices_of_a_projection_are_read_in_place(recorder, dtype, width):
    """q, k and v as slices of one projection keep its row as their stride; rows that are not 16 bytes
    apart are copied."""
    proj = meta(2, 5, 2 * 2 * 8 + 4 * 16 + 4 * width, dtype=dtype)
    q, k = (proj[..., 16 * i:16 * i + 16].unflatten(-1, (2, 8)) for i in (0, 1))
    v = proj[..., 32:96].unflatten(-1, (4, 16))
    gdn.linear_attention(q, k, v, meta(4))
    d = recorder.calls[0][1]
    assert (d.q_stride, d.k_stride, d.v_stride) == (proj.shape[-1],) * 3 and d.head_decay == 1
    odd = meta(2, 5, 2 * 2 * 8 + 4 * 16 + 1, dtype=dtype)
    gdn.linear_attention(odd[..., :16].unflatten(-1, (2, 8)), k, v, meta(4))
    assert recorder.calls[1][1].q_stride == 0 and recorder.calls[1][1].v_stride == proj.shape[-1]


def test_rows_of_the_block_norm_are_read_in_place(recorder):
    wide = meta(3, 5, 40)
    gdn.block_norm(meta(3, 5, 8), wide[..., 8:16], gate=wide[..., 16:24])
    d = recorder.calls[0][1]
    assert (d.rows, d.channels, d.h_stride, d.gate_stride) == (15, 8, 40, 40)
