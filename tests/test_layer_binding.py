"""What the Python binding hands to the library, on the host (no GPU needed): meta tensors of any
size, and a library that records its calls instead of launching."""
import contextlib

import pytest
import torch

import gated_deltanet_chunked_02_amd as gdn

BF16, F32 = torch.bfloat16, torch.float32


def meta(*shape, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="meta")


class Recorder:
    """The library's host-only queries, and its launches recorded as (name, arguments)."""

    def __init__(self, lib):
        self.lib, self.calls, self.device = lib, [], 0

    def __getattr__(self, name):
        if name.endswith("_size") or name == "gdn_status_string":
            return getattr(self.lib, name)

        def call(*args):
            # descriptors are passed by reference
            self.calls.append((name, getattr(args[0], "_obj", args[0]), args[1:], self.device))
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    rec = Recorder(gdn.load())

    @contextlib.contextmanager
    def device(d):
        before, rec.device = rec.device, d
        yield
        rec.device = before

    for module in (gdn, gdn.ssm):
        monkeypatch.setattr(module, "load", lambda: rec)
        monkeypatch.setattr(module, "_check_devices", lambda *a: None)
    monkeypatch.setattr(gdn, "_raw", (lambda: 0, lambda index: 0))
    monkeypatch.setattr(torch.cuda, "device", device)
    return rec


def scan_args(B, T, C=8, G=1, S=4):
    return (meta(B, T, C), meta(B, T, C), meta(C, S), meta(B, T, G, S), meta(B, T, G, S))


def step_args(n, lines, C=8, G=1, S=4):
    return (meta(lines, C, S), meta(n, C), meta(n, C), meta(C, S), meta(n, G, S), meta(n, G, S))


BIG = 2 ** 32 + 5


@pytest.mark.parametrize("call", [
    lambda: gdn.selective_scan(*scan_args(1, BIG)),
    lambda: gdn.selective_scan(*scan_args(BIG, 1)),
    lambda: gdn.selective_scan(*scan_args(1, 1, C=2 ** 32 + 8)),
    lambda: gdn.selective_scan(*scan_args(1, 3), cu_seqlens=meta(BIG, dtype=torch.int32)),
    lambda: gdn.selective_scan_bwd(*scan_args(1, BIG), meta(1, BIG, 8)),
    lambda: gdn.selective_state_update(*step_args(BIG, BIG)),
    lambda: gdn.selective_state_update(*step_args(2, BIG)),
    lambda: gdn.causal_conv1d(meta(1, BIG, 8), meta(8, 4)),
    lambda: gdn.causal_conv1d(meta(1, 4, 8), meta(8, 4), conv_state=meta(BIG, 3, 8)),
    lambda: gdn.causal_conv1d_bwd(meta(1, BIG, 8), meta(8, 4), meta(1, BIG, 8)),
    lambda: gdn.group_norm(meta(1, BIG, 8), 2),
    lambda: gdn.group_norm(meta(1, 2 ** 16, 2 ** 16, 8), 2),
    lambda: gdn.group_norm(meta(BIG, 8), 2),
    lambda: gdn.group_norm_bwd(meta(1, BIG, 8), meta(1, BIG, 8), 2, meta(1, 2), meta(1, 2)),
    lambda: gdn.chunk_gated_delta_rule(meta(1, BIG, 1, 64), meta(1, BIG, 1, 64),
                                       meta(1, BIG, 1, 64), meta(1, BIG, 1), meta(1, BIG, 1)),
])
def test_sizes_past_32_bits_are_refused(recorder, call):
    """A descriptor's fields have 32 bits; a larger size must not come out as a small one."""
    with pytest.raises(gdn.GdnError) as e:
        call()
    assert e.value.status == 2 and not recorder.calls


def _gdn_args(T=2, D=64):
    return (meta(1, T, 1, D), meta(1, T, 1, D), meta(1, T, 1, D))


@pytest.mark.parametrize("name,call", [
    ("gdn_selective_scan_fwd", lambda: gdn.selective_scan(*scan_args(1, 5))),
    ("gdn_selective_scan_bwd", lambda: gdn.selective_scan_bwd(*scan_args(1, 5), meta(1, 5, 8))),
    ("gdn_selective_state_update", lambda: gdn.selective_state_update(*step_args(2, 3))),
    ("gdn_causal_conv1d_fwd", lambda: gdn.causal_conv1d(meta(1, 5, 8), meta(8, 4))),
    ("gdn_causal_conv1d_bwd", lambda: gdn.causal_conv1d_bwd(meta(1, 5, 8), meta(8, 4),
                                                            meta(1, 5, 8))),
    ("gdn_group_norm_fwd", lambda: gdn.group_norm(meta(3, 8), 2)),
    ("gdn_group_norm_bwd", lambda: gdn.group_norm_bwd(meta(3, 8), meta(3, 8), 2, meta(3, 2),
                                                      meta(3, 2))),
    ("gdn_chunk_fwd", lambda: gdn.chunk_gated_delta_rule(*_gdn_args(), meta(1, 2, 1),
                                                         meta(1, 2, 1))),
    ("gdn_chunk_bwd", lambda: gdn.chunk_gated_delta_rule_bwd(*_gdn_args(), meta(1, 2, 1),
                                                             meta(1, 2, 1), meta(1, 2, 1, 64))),
    ("gdn_fused_sigmoid_gating_delta_rule", lambda: gdn.fused_sigmoid_gating_delta_rule(
        *_gdn_args(), meta(1, 2, 1), meta(1, 2, 1), meta(1))),
])
def test_launches_with_the_tensors_device_current(recorder, name, call):
    """Device 0 is current; the tensors are on another one, whose default stream is 0 as well."""
    call()
    assert [(c[0], c[3]) for c in recorder.calls] == [(name, torch.device("meta"))]
    assert recorder.device == 0


def test_64_bit_lines_outside_the_pool_stay_outside():
    from gated_deltanet_chunked_02_amd.ssm import _indices
    given = torch.tensor([0, 5, -1, -7, 2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 31 - 1])
    got = _indices("cache_indices", given, 9)
    assert got.dtype == torch.int32 and got[:2].tolist() == [0, 5]
    assert all(i < 0 or i == 2 ** 31 - 1 for i in got[2:].tolist())
    assert _indices("cache_indices", got, 9) is got
