"""Newton-Schulz orthogonalisation on the GPU against 64 bits."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

from . import mx_util as mx

pytestmark = pytest.mark.gpu
A = 3.4445


def grads(g, B, M, N, dtype):
    """Low-rank gradients under noise."""
    r = min(M, N, 16)
    low = torch.randn(B, M, r, generator=g) @ (torch.randn(B, r, N, generator=g) / torch.arange(1, r + 1)[:, None])
    return (1e-3 * (low + torch.randn(B, M, N, generator=g))).to(dtype)


def check(got, want, dtype, steps=5):
    """In the Frobenius norm: the output's own rounding (half a step), and the roundings of the factors. Those are
    half a step of 16 bits (2^-17), of X and of P in each step; the first has norm 2^-17 |X| = 2^-17 and is multiplied by
    at most a in each of `steps` steps, the later ones by less (their sum is taken as as much again)."""
    off = torch.linalg.vector_norm(got.double().cpu() - want)
    norm = torch.linalg.vector_norm(want)
    tol = mx.half_step(dtype) * norm + 2 * 2.0 ** -17 * A ** steps
    assert off <= tol, f"off by {off / norm:.3g} of the norm, {tol / norm:.3g} allowed"


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("B,M,N", [(1, 1, 1), (2, 1, 70), (1, 70, 1), (3, 5, 3), (1, 64, 64), (2, 65, 63), (1, 128, 128),
                                   (1, 129, 200), (2, 300, 190), (1, 100, 1000), (1, 1000, 100), (1, 640, 700), (5, 256, 512)])
def test_against_64_bits(B, M, N, name):
    dt = mx.TYPES[name]
    g = torch.Generator()
    g.manual_seed(B + M + N)
    x = grads(g, B, M, N, dt)
    got = mp.newton_schulz(x.cuda())
    assert got.dtype == dt and got.shape == x.shape
    for b in range(B):
        check(got[b], mx.newton_schulz(x[b]), dt)
        one = mp.newton_schulz(x[b].cuda())
        assert torch.equal(one, got[b])   # a matrix does not depend on its batch


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 6, 7])
@pytest.mark.parametrize("M,N", [(96, 160), (200, 72), (60, 500)])
def test_steps(steps, M, N):
    g = torch.Generator()
    g.manual_seed(steps)
    x = grads(g, 1, M, N, torch.float16)[0]
    check(mp.newton_schulz(x.cuda(), steps=steps), mx.newton_schulz(x, steps=steps), torch.float16, steps)


def test_singular_values():
    """With more steps and the classical coefficients the singular values go to one."""
    g = torch.Generator()
    g.manual_seed(1)
    x = torch.randn(192, 256, generator=g).to(torch.bfloat16)
    y = mp.newton_schulz(x.cuda(), steps=24, coeffs=(1.875, -1.25, 0.375)).double().cpu()
    s = torch.linalg.svdvals(y)
    # bf16 outputs: a rounding matrix of entries up to 2^-9 |y|, |y|_F = sqrt(192)
    assert (s - 1).abs().max() <= 2.0 ** -9 * 192 ** 0.5


def test_views_in_place_and_strides():
    g = torch.Generator()
    g.manual_seed(2)
    base = grads(g, 3, 90, 150, torch.bfloat16).cuda()
    x = base[:, 7:80, 3:140]
    want = mp.newton_schulz(x.contiguous())
    out = torch.full((3, 90, 150), 5.0, dtype=torch.bfloat16, device="cuda")
    mp.newton_schulz(x, out=out[:, 7:80, 3:140])
    assert torch.equal(out[:, 7:80, 3:140], want)
    out[:, 7:80, 3:140] = 5
    assert (out == 5).all()
    mp.newton_schulz(x, out=x)
    assert torch.equal(x, want)
    # one matrix for the whole batch
    m = grads(g, 1, 40, 50, torch.bfloat16).cuda()
    y = mp.newton_schulz(m.expand(4, 40, 50))
    assert torch.equal(y, mp.newton_schulz(m).expand(4, 40, 50))


def test_zeros_infinities_and_scale():
    z = torch.zeros(2, 70, 90, dtype=torch.bfloat16, device="cuda")
    z[1] = torch.randn(70, 90, device="cuda")
    y = mp.newton_schulz(z)
    assert not y[0].any() and torch.isfinite(y[1]).all()
    z[0, 3, 4] = float("inf")
    y2 = mp.newton_schulz(z)
    assert torch.isnan(y2[0]).all() and torch.equal(y2[1], y[1])
    z[0] = 0
    z[0, 5, 5] = float("nan")
    assert torch.isnan(mp.newton_schulz(z)[0]).all()
    # the scale of the input drops out (powers of two: the same bits)
    x = torch.randn(80, 64, device="cuda").to(torch.bfloat16)
    assert torch.equal(mp.newton_schulz(x, eps=0.0), mp.newton_schulz(x * 2.0 ** -30, eps=0.0))
    check(mp.newton_schulz(x * 2.0 ** 20), mx.newton_schulz(x.cpu()), torch.bfloat16)


def test_empty_and_graph():
    e = torch.empty(0, 4, 5, dtype=torch.float16, device="cuda")
    assert mp.newton_schulz(e).shape == (0, 4, 5)
    assert mp.newton_schulz(e.new_empty((3, 0, 5))).shape == (3, 0, 5)
    x = torch.randn(2, 130, 200, device="cuda").half()
    mp.newton_schulz(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mp.newton_schulz(x)
    for _ in range(4):
        x.copy_(torch.randn(2, 130, 200).half())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mp.newton_schulz(x))
