"""Trains one linear layer in MXFP4: forward and backward products on 4-bit operands, an orthogonalised momentum update
of the weight, and the weight quantised again in both orientations.

    python examples/mxfp4_layer.py [--steps 60] [--tokens 512] [--out 384] [--in 256]

The layer learns a fixed random map from noisy samples; the loss, printed every ten steps, falls towards the error of
the 4-bit forward pass.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import precision_dense_gemm_tiled_amd as mp  # noqa: E402


class Layer:
    """Y = X W^T + bias with W in MXFP4 for the products, in fp32 for the update."""

    def __init__(self, out_features, in_features, lr=0.02, momentum=0.9):
        self.weight = torch.randn(out_features, in_features, device="cuda") / in_features ** 0.5
        self.bias = torch.zeros(out_features, device="cuda", dtype=torch.bfloat16)
        self.m = torch.zeros_like(self.weight)
        self.lr, self.momentum = lr, momentum
        self.hold()

    def hold(self):
        self.wq, self.ws, self.wtq, self.wts = mp.quantize_mxfp4_both(self.weight.bfloat16())

    def forward(self, x):
        # X^T is for the weight's gradient; without a backward pass gemm_mxfp4_dyn(x, ...) quantises X in the product
        xq, xs, *self.xt = mp.quantize_mxfp4_both(x)
        return mp.gemm_mxfp4(xq, xs, self.wq, self.ws, x.shape[1], bias=self.bias, dtype=x.dtype)

    def backward(self, dy):
        return mp.gemm_mxfp4_backward(dy, self.wtq, self.wts, *self.xt)

    def update(self, dw):
        self.m.mul_(self.momentum).add_(dw)
        step = mp.newton_schulz(self.m.bfloat16())
        self.weight.sub_(step.float(), alpha=self.lr * max(1.0, self.weight.shape[0] / self.weight.shape[1]) ** 0.5)
        self.hold()


def train(steps=60, tokens=512, out_features=384, in_features=256, seed=0, show=print):
    """Trains and returns the losses."""
    torch.manual_seed(seed)
    target = torch.randn(out_features, in_features, device="cuda") / in_features ** 0.5
    layer = Layer(out_features, in_features)
    losses = []
    for k in range(steps):
        layer.lr = 0.2 * (1 - k / steps)   # (every singular direction moves by lr: together further than the maps are apart)
        x = torch.randn(tokens, in_features, device="cuda").bfloat16()
        want = x.float() @ target.t()
        y = layer.forward(x)
        off = y.float() - want
        losses.append((off.square().sum() / want.square().sum()).item())
        _, dw = layer.backward((off * (2 / tokens)).bfloat16())
        layer.update(dw)
        if k % 10 == 0 or k == steps - 1:
            show(f"step {k:3d}  relative squared error {losses[-1]:.4f}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--out", type=int, default=384)
    ap.add_argument("--in", dest="inp", type=int, default=256)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.out, a.inp)


if __name__ == "__main__":
    main()
