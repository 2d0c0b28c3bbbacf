"""The example layer learns: forward, backward, update and quantisation together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_the_layer_learns():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_layer.py")
    spec = importlib.util.spec_from_file_location("mxfp4_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=60, tokens=300, out_features=200, in_features=136, show=lambda s: None)
    # two independent maps of the same size: about 2 at the start. e2m1 keeps a value to a relative 1/8 rms or
    # better, X and W each: well under 0.1 in the square at the end
    assert 1.5 < losses[0] < 2.5
    assert losses[-1] < 0.1
