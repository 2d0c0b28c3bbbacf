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


def dual(x):
    return torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))


def calls(mp):
    """Every call with its floating-point operands: what takes X, and the operands' shapes."""
    h = lambda r, c: torch.zeros(r, c, dtype=torch.float16)   # noqa: E731
    q, s = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    u8, sc = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    back = [h(4, 8), h(4, 64), h(8, 64), h(8, 64), h(4, 8), h(4, 8)]
    return {"quantize_i8": (mp.quantize_i8, [h(4, 64)]), "dequantize_i8": (mp.dequantize_i8, [q, s]),
            "gemm_w8a8": (mp.gemm_w8a8, [q, s, q, s.clone()]), "gemm_w8a8_dyn": (mp.gemm_w8a8_dyn, [h(4, 64), q, s]),
            "gemm_gated": (mp.gemm_gated, [h(4, 64), h(8, 64), h(8, 64)]), "gemm_gated_backward": (mp.gemm_gated_backward, back),
            "gemm_gated_w8a8": (mp.gemm_gated_w8a8, [q, s, q, s, q, s]), "gemm_gated_w8a8_dyn": (mp.gemm_gated_w8a8_dyn, [h(4, 64), q, s, q, s]),
            "gemm_mxfp4_dyn": (mp.gemm_mxfp4_dyn, [h(4, 64), u8, sc]), "gemm_mxfp4_backward": (mp.gemm_mxfp4_backward, [h(4, 8), u8, sc, u8, sc]),
            "newton_schulz": (mp.newton_schulz, [h(4, 64)])}


@pytest.mark.parametrize("name", ["quantize_i8", "dequantize_i8", "gemm_w8a8", "gemm_w8a8_dyn", "gemm_gated", "gemm_gated_backward", "gemm_gated_w8a8",
                                  "gemm_gated_w8a8_dyn", "gemm_mxfp4_dyn", "gemm_mxfp4_backward", "newton_schulz"])
def test_a_lost_tangent_raises(mp, name):
    f, args = calls(mp)[name]
    at = next(i for i, v in enumerate(args) if v.is_floating_point())

    def call(v):
        return f(*args[:at], v, *args[at + 1:])

    with torch.autograd.forward_ad.dual_level():
        for grad in (torch.enable_grad(), torch.no_grad()):   # (torch keeps tangents under no_grad)
            with grad, pytest.raises(RuntimeError, match="tangent.*autograd"):
                call(dual(args[at]))
        # where torch itself drops tangents, as inside an autograd.Function, there is nothing to lose
        with torch.autograd.forward_ad._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="device|not on"):
            call(dual(args[at]))
        with pytest.raises(ValueError, match="device|not on"):
            call(args[at])
