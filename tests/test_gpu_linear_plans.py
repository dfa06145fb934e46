"""Linear attention's calls with states in the caller's own buffers: the same bits wherever the initial
and final states (the gradients of both) are held, in every way of running a batch."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

PLANS = [
    # T, lens, H, Hg: split sequences, short ones, whole ones (a head a CU), packed in segments
    (900, None, 4, 2), (100, None, 4, 2), (900, None, 256, 64),
    (1400, (0, 700, 3, 1, 696), 4, 4), (1400, (0, 700, 3, 1, 696), 300, 300), (300, (0, 300), 2, 1)]


def setup(T, lens, H, Hg, dtype, head):
    import gated_deltanet_chunked_02_amd as gdn
    r = torch.Generator().manual_seed(T + H)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    N = len(lens) if lens else 1
    t = dict(q=n(1, T, Hg, 32).to(dtype), k=n(1, T, Hg, 32).to(dtype), v=n(1, T, H, 40).to(dtype),
             g=-torch.rand(H if head else 1, generator=r) if head
             else -torch.rand(1, T, H, generator=r),
             do=n(1, T, H, 40).to(dtype), h0=n(N, H, 32, 40), dht=n(N, H, 32, 40))
    t = {x: y.cuda() for x, y in t.items()}
    t["cu"] = torch.tensor((0,) + lens).cumsum(0).int().cuda() if lens else None
    desc = gdn.GdnLinearDesc(1, T, N, H, Hg, 32, 40, 1 if dtype == torch.bfloat16 else 0, int(head), 0,
                             0.2, 0, 0, 0, None, 0)
    return gdn, t, desc


def space(desc, need):
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    desc.workspace, desc.workspace_bytes = ctypes.c_void_p(ws.data_ptr()), ws.numel()
    return ws


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,lens,H,Hg", PLANS)
def test_states_in_one_buffer(T, lens, H, Hg, dtype, head):
    gdn, t, desc = setup(T, lens, H, Hg, dtype, head)
    ws = space(desc, gdn.gdn_linear_attn_workspace_size(desc))
    args = (t["q"], t["k"], t["v"], t["g"])
    o, ht, o2, both = (torch.empty_like(x) for x in (t["v"], t["h0"], t["v"], t["h0"]))
    both.copy_(t["h0"])
    assert gdn.gdn_linear_attn_fwd(desc, *args, t["h0"], t["cu"], o, ht) == 0
    ws.fill_(255)  # what an earlier call left is not used
    assert gdn.gdn_linear_attn_fwd(desc, *args, both, t["cu"], o2, both) == 0
    assert torch.equal(o, o2) and torch.equal(ht, both)
    if lens:  # a sequence of no tokens hands its state through
        assert torch.equal(ht[0], t["h0"][0])

    ws = space(desc, gdn.gdn_linear_attn_bwd_workspace_size(desc))
    one, two = ([torch.empty_like(t[x]) for x in ("q", "k", "v", "g", "dht")] for _ in range(2))
    two[4].copy_(t["dht"])
    assert gdn.gdn_linear_attn_bwd(desc, *args, t["h0"], t["cu"], t["do"], t["dht"], *one) == 0
    ws.fill_(255)
    assert gdn.gdn_linear_attn_bwd(desc, *args, t["h0"], t["cu"], t["do"], two[4], *two) == 0
    for i, (a, b) in enumerate(zip(one, two)):
        assert torch.equal(a, b), i
    if lens:
        assert torch.equal(one[4][0], t["dht"][0])


def test_step_on_a_pool_past_2_to_31_elements():
    """Lines on either side of 2^31 and 2^32 elements (and bytes) of the pool."""
    import gated_deltanet_chunked_02_amd as gdn
    H, D = 32, 128
    lines = (1 << 32) // (H * D * D) + 3
    r = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=r, device="cuda")  # noqa: E731
    at = [0, (1 << 31) // (H * D * D), lines - 2]
    pool = torch.empty(lines, H, D, D, device="cuda")
    small = n(3, H, D, D)
    for i, line in enumerate(at):
        pool[line] = small[i]
    q, k, v = (n(3, H, D).bfloat16() for _ in range(3))
    g = -torch.rand(3, H, generator=r, device="cuda")
    read = torch.tensor(at, dtype=torch.int32, device="cuda")
    write = torch.tensor([lines - 1, at[1], 1], dtype=torch.int32, device="cuda")
    o = gdn.linear_state_update(pool, q, k, v, g, cache_indices=read, out_indices=write)
    want = gdn.linear_state_update(small, q, k, v, g)
    assert torch.equal(o, want)
    for i, line in enumerate((lines - 1, at[1], 1)):
        assert torch.equal(pool[line], small[i]), line
