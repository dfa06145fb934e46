"""How linear attention runs a batch: its launches, and the same results on either side of each choice."""
import pytest
import torch

from test_gpu_linear import TOL, TOL_F32, check, dev, make, oracle_fwd, run_fwd

pytestmark = pytest.mark.gpu


def kernels(run):
    """Kernels of a call, by the nodes of a graph that captured it."""
    import ctypes
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        run()
    with open("/proc/self/maps") as f:
        path = next(x.split()[-1] for x in f if "libamdhip64" in x)
    count = ctypes.c_size_t(0)
    nodes = ctypes.CDLL(path).hipGraphGetNodes
    assert nodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(count)) == 0
    return count.value


@pytest.mark.parametrize("T,H,D,launches", [
    # short sequences whole; 16 segments make their start states themselves, more a launch composes
    (300, 1, 8, 1), (1024, 2, 32, 2), (2048, 2, 32, 2), (2176, 2, 32, 3), (4096, 4, 64, 3),
    (16384, 1, 8, 3), (1024, 1, 128, 2), (1152, 1, 128, 3), (100, 4, 64, 1)])
def test_many_segments_are_composed_by_a_launch(T, H, D, launches):
    import gated_deltanet_chunked_02_amd as gdn
    p = make(1, T, H, H, D, D, "bf16", seed=T)
    q = dev(p)
    args = (q["q"], q["k"], q["v"], q["g"])
    assert kernels(lambda: gdn.linear_attention(*args, initial_state=q["h0"])) == launches
    if T <= 4096:
        o_ref, ht_ref = oracle_fwd(p)
        o, ht = run_fwd(p)
        check("o", o, o_ref, TOL["bf16"])
        check("ht", ht, ht_ref, TOL_F32)
