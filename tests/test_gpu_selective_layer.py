"""The example layer, which runs the state-space calls together as a model does."""
import os
import sys

import pytest

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
