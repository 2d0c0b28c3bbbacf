"""Newton-Schulz orthogonalisation against 64 bits where roundings grow: exactly low-rank matrices, several steps in
a group, small matrices and many steps.

The tolerance, in the Frobenius norm. The output's rounding is half a step. A step stores four matrices (A, Q, T or
W, X) in 22 bits, each off by at most 2^-22 of itself, and sums in fp32; what the first steps leave in a direction
is lifted by a at every step, like a signal there, until it has grown to the size of the others. Of an error spread
evenly over the m directions, direction i is lifted by g_i = min(a^steps, 1.21 / s_i), s_i being the singular value
of G / |G| and 1.21 the most that the polynomial leaves of [0, 1.21]; in all that is the root mean square of the g_i.
The steps' errors make a geometric series, 4 a / (a - 1) < 8 times the first's. Every step leaves as much of its own
on a result of norm |Y|. So half a step of |Y|, and 2^-19 (rms g + steps |Y|)."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

from . import mx_util as mx

pytestmark = pytest.mark.gpu
A, MOST = 3.4445, 1.21


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def check(x, steps=5):
    """x: a CPU matrix. Returns the kernel's output."""
    got = mp.newton_schulz(x.cuda(), steps=steps)
    want = mx.newton_schulz(x, steps=steps)
    off, norm = torch.linalg.vector_norm(got.double().cpu() - want), torch.linalg.vector_norm(want)
    s = torch.linalg.svdvals(x.double())
    s = torch.where(s > 1e-12 * s[0], s, torch.zeros_like(s)) / torch.linalg.vector_norm(s)
    lift = torch.minimum(torch.full_like(s, A ** steps), MOST / s.clamp(min=1e-30)).square().mean().sqrt()
    tol = mx.half_step(x.dtype) * norm + 2.0 ** -19 * (lift + steps * norm)
    assert off <= tol, f"off by {off / norm:.3g} of the norm, {tol / norm:.3g} allowed"
    return got


def low_rank(M, N, r, dtype):
    """Products of small whole numbers: rank r exactly, also in 16 bits."""
    g = gen(M + N + r)
    return (torch.randint(-3, 4, (M, r), generator=g).float() @ torch.randint(-3, 4, (r, N), generator=g).float()).to(dtype)


SMALL = [(64, 64), (40, 70), (100, 1000), (128, 128), (900, 128)]
LARGE = [(256, 256), (200, 1000), (1000, 300), (129, 600)]


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("steps", [2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("r", [1, 4])
@pytest.mark.parametrize("M,N", SMALL + LARGE)
def test_exactly_low_rank(M, N, r, steps, name):
    check(low_rank(M, N, r, mx.TYPES[name]), steps)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("M,N", SMALL + LARGE)
def test_many_steps_of_low_rank(M, N, name):
    """Roundings have become singular values like the others, all of them within the polynomial's bound."""
    y = mp.newton_schulz(low_rank(M, N, 4, mx.TYPES[name]).cuda(), steps=12).double().cpu()
    m = min(M, N)
    # (the rounding of the output: a matrix of entries of half a step of |y|, of norm at most that of y, sqrt(m) MOST)
    assert torch.linalg.matrix_norm(y, 2) <= MOST * (1 + mx.half_step(mx.TYPES[name]) * m ** 0.5)


def grads(g, M, N, dtype, noise=1.0, rank=16):
    r = min(M, N, rank)
    low = torch.randn(M, r, generator=g) @ torch.randn(r, N, generator=g)
    return (1e-3 * (low + noise * torch.randn(M, N, generator=g))).to(dtype)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 70), (70, 1), (5, 3), (2, 2), (17, 33), (64, 64), (65, 63), (128, 128), (129, 200),
                                 (300, 190), (100, 1000), (1000, 100), (640, 700), (256, 512)])
def test_sizes(M, N, name):
    check(grads(gen(M + N), M, N, mx.TYPES[name]))


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 6, 7])
@pytest.mark.parametrize("M,N", [(96, 160), (200, 72), (60, 500), (5, 3), (150, 170), (160, 700)])
def test_steps(steps, M, N):
    check(grads(gen(steps), M, N, torch.float16), steps)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("steps", [4, 5, 7])
@pytest.mark.parametrize("noise", [1e-2, 1e-4])
@pytest.mark.parametrize("M,N", [(64, 64), (128, 128), (100, 1000), (256, 256), (256, 1024)])
def test_rank_one_under_noise(M, N, noise, steps, name):
    check(grads(gen(M + N), M, N, mx.TYPES[name], noise=noise, rank=1), steps)
