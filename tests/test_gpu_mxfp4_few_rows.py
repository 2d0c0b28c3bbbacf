"""MXFP4 products of few rows at the widths and lengths where their kernels change, against 64 bits."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

from . import mx_util as mx

pytestmark = pytest.mark.gpu


def run(M, N, K, dtype):
    g = torch.Generator()
    g.manual_seed(M + 3 * N + 5 * K)
    A, B = mx.random_held(g, M, K, spread=1), mx.random_held(g, N, K, spread=1)
    bias = torch.randn(N, generator=g).to(dtype)
    a, b = mx.values(*A, K), mx.values(*B, K)
    y, t = a @ b.t() + bias.double(), a.abs() @ b.abs().t() + bias.double().abs()
    got = mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), K, bias=bias.cuda(), dtype=dtype)
    mx.check(got, y, mx.gemm_tol(y, t, (K + 31) // 32, dtype))
    x = (0.1 * torch.randn(M, K, generator=g)).to(dtype)
    X = mx.on_gpu(mx.quantize(x))
    assert torch.equal(mp.gemm_mxfp4_dyn(x.cuda(), *mx.on_gpu(B), bias=bias.cuda()),
                       mp.gemm_mxfp4(*X, *mx.on_gpu(B), K, bias=bias.cuda(), dtype=dtype))


# 16 and 32 columns per workgroup: up to four rows from 8192 columns on, with more from 4097 on
@pytest.mark.parametrize("M", [1, 4, 5, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(4096, 520), (4097, 1056), (6000, 264), (8191, 520), (8192, 96)])
def test_widths(M, N, K):
    run(M, N, K, torch.bfloat16)


# tiles instead of the skinny kernel where rows times K is large, on both sides of that
@pytest.mark.parametrize("M,N,K", [(16, 200, 16416), (17, 300, 16384), (24, 130, 16640), (25, 130, 16640), (32, 4100, 12480),
                                   (32, 100, 12544), (33, 2048, 16384), (64, 1000, 6240), (64, 1000, 6272), (64, 33, 9000)])
@pytest.mark.parametrize("name", ["f16", "f32"])
def test_long_rows(M, N, K, name):
    run(M, N, K, mx.TYPES[name])
