"""On the device: an argument of a floating-point call that requires grad raises, under no_grad the call runs."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

pytestmark = pytest.mark.gpu


def test_bias_out_and_weights():
    w = torch.randn(48, 64, device="cuda", requires_grad=True)
    q, s = mp.quantize_mxfp4(w)   # codes: no gradient to lose
    x = torch.randn(5, 64, device="cuda")
    bias = torch.zeros(48, device="cuda", requires_grad=True)
    xq, xs = mp.quantize_mxfp4(x)
    want = mp.gemm_mxfp4_dyn(x, q, s)
    out = torch.empty(5, 48, device="cuda", requires_grad=True)
    for call in (lambda: mp.gemm_mxfp4_dyn(x, q, s, bias=bias), lambda: mp.gemm_mxfp4(xq, xs, q, s, 64, bias=bias),
                 lambda: mp.gemm_mxfp4_dyn(x, q, s, out=out), lambda: mp.dequantize_mxfp4(xq, xs, 64, out=torch.empty_like(x).requires_grad_())):
        with pytest.raises(RuntimeError, match="autograd"):
            call()
        with torch.no_grad():
            call()
    assert torch.equal(out, want)
