"""The example layer quantises a batch of activations once."""
import importlib.util
import os

import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

pytestmark = pytest.mark.gpu


def test_one_quantisation_per_batch():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_layer.py")
    spec = importlib.util.spec_from_file_location("mxfp4_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(200, 136)
    layer.bias.normal_()
    x = torch.randn(70, 136, device="cuda").bfloat16()
    called = []

    class Recorder:
        def __getattr__(self, name):
            def call(*a, **k):
                called.append(name)
                return getattr(mp, name)(*a, **k)
            return call

    example.mp = Recorder()
    y = layer.forward(x)
    assert called == ["quantize_mxfp4_both", "gemm_mxfp4"]   # (gemm_mxfp4_dyn would quantise x again)
    assert torch.equal(y, mp.gemm_mxfp4_dyn(x, layer.wq, layer.ws, bias=layer.bias))
    dx, dw = layer.backward(torch.randn(70, 200, device="cuda").bfloat16())
    assert dx.shape == x.shape and dw.shape == (200, 136) and called[2:] == ["gemm_mxfp4_backward"]
