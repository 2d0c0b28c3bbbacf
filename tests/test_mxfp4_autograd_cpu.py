"""The MXFP4 and Newton-Schulz calls stay outside autograd and say so where a gradient would be lost. (Host tensors:
the check comes before the one for the device, whose ValueError shows that the first has passed.)"""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    if not os.path.exists(mp.calls_path):
        from precision_dense_gemm_tiled_amd import build
        build.build()
    return mp


def calls(mp):
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    x = lambda: torch.zeros(4, 64, dtype=torch.float16)   # noqa: E731
    return {"dyn X": (x, lambda t: mp.gemm_mxfp4_dyn(t, q, s)),
            "backward dY": (x, lambda t: mp.gemm_mxfp4_backward(t, q, s, q, s)),
            "newton_schulz G": (x, lambda t: mp.newton_schulz(t)),
            "newton_schulz out": (x, lambda t: mp.newton_schulz(x(), out=t))}


@pytest.mark.parametrize("name", ["dyn X", "backward dY", "newton_schulz G", "newton_schulz out"])
def test_a_lost_gradient_raises(mp, name):
    make, call = calls(mp)[name]
    with pytest.raises(RuntimeError, match="autograd"):
        call(make().requires_grad_())
    with pytest.raises(ValueError):
        call(make())
    with pytest.raises(ValueError):
        call(make().requires_grad_().detach())
    with torch.no_grad(), pytest.raises(ValueError):
        call(make().requires_grad_())


def test_inside_a_function(mp):
    """An autograd.Function's own passes run without grad mode, so they may call."""
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)

    class F(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            with pytest.raises(ValueError):
                mp.gemm_mxfp4_dyn(x, q, s)
            return x * 1

        @staticmethod
        def backward(ctx, dy):
            with pytest.raises(ValueError):
                mp.gemm_mxfp4_backward(dy, q, s, q, s)
            return dy

    F.apply(torch.zeros(4, 64, dtype=torch.float16, requires_grad=True)).sum().backward()


def test_quantisation_of_a_weight_that_requires_grad(mp):
    with pytest.raises(ValueError):
        mp.quantize_mxfp4(torch.zeros(4, 64, requires_grad=True))
