"""Derivatives that a call of the integer layer or of the gated block would lose are refused, without a GPU: the refusal
comes before the tensors' device is looked at."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    if not os.path.exists(mp.lib_path) or not os.path.exists(mp.calls_path):
        from precision_dense_gemm_tiled_amd import build
        build.build()
    return mp


def test_quantising_loses_no_gradient(mp):
    """The scales that quantize_i8 returns are a function of X, and so is what is computed from them."""
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        x = torch.zeros(4, 64, dtype=dt)
        with pytest.raises(RuntimeError, match="X requires grad.*autograd"):
            mp.quantize_i8(x.clone().requires_grad_())
        with pytest.raises(RuntimeError, match="X requires grad.*autograd"):
            mp.quantize_i8(x.clone().requires_grad_() * 2)
        for y in (x, x.clone().requires_grad_().detach()):
            with pytest.raises(ValueError, match="device tensor"):
                mp.quantize_i8(y)
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            mp.quantize_i8(x.clone().requires_grad_())
