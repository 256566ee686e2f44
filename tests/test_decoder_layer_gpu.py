"""The example that trains one decoder layer: norm, aggregation and attention
together, with gradients through all of them."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_decoder_layer_learns():
    import decoder_layer

    import deformable_view_feature_gb300 as da
    da.build.build()
    losses, layer = decoder_layer.train(steps=6, small=True, lr=1.0)
    assert losses[-1] < losses[0]
    for name, p in layer.named_parameters():
        assert bool(torch.isfinite(p.grad).all()) and bool(p.grad.any()), name
    assert not da.waits_gave_up()
