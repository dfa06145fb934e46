"""Where linear attention cuts sequences into segments, on the host (no GPU needed): read off the workspace
that its calls ask for."""
import pytest

from test_layer_refusals import size
from test_linear_refusals import SIZES, linear_desc


def segments(B, T, N, H):
    """Segments of a batch's forward (0: whole sequences), by the states of 64 x 64 kept for them."""
    status, need = size(SIZES[0], linear_desc(B=B, T=T, N=N, H=H, Hg=H))
    assert status == 0
    return need // (H * 64 * 64 * 4)


@pytest.mark.parametrize("pairs,cut", [(64, True), (128, True), (160, True), (170, True),
                                       (180, False), (192, False), (224, False), (255, False),
                                       (256, False), (257, False), (288, False), (512, False)])
def test_dense_batches_are_cut_where_three_segments_fit(pairs, cut):
    for B in range(1, 9):
        if pairs % B == 0:
            assert (segments(B, 2048, B, pairs // B) >= 3 * B) == cut
            assert cut or segments(B, 2048, B, pairs // B) == 0


def test_packed_batches_have_no_step_at_a_head_a_cu():
    """Eight sequences: segments get fewer with the heads, evenly, to 288 pairs."""
    counts = [segments(1, 12454, 8, H) for H in range(24, 37)]
    assert all(b <= a <= b + 3 for a, b in zip(counts, counts[1:])), counts
    assert counts[-1] > 2 * 8


def test_packed_gradients_come_to_the_mean_evenly():
    """To 512 pairs, where as many segments as fill the GPU are twice the mean length."""
    def at(H):
        # two states a segment; what is kept for the gradient comes on top, by length alone
        return size(SIZES[1], linear_desc(B=1, T=16384, N=8, H=H, Hg=H))[1] // (H * 64 * 64 * 4)
    sizes = [at(H) for H in range(24, 65)]
    assert all(b <= a for a, b in zip(sizes, sizes[1:]))
    assert sizes[-1] == at(65) == at(100)
