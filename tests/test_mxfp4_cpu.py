"""MXFP4 and Newton-Schulz without a GPU: the test's own quantiser on worked
values, refusals (the handle is checked last, so a NULL handle reaches every
check) and the scratch sizes."""
import os

import pytest
import torch

from . import mx_util as mx

INVALID, UNSUPPORTED = 1, 2
P = 1 << 20   # an address that is only ever checked


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    if not os.path.exists(mp.lib_path):
        from precision_dense_gemm_tiled_amd import build
        build.build()
    mp.lib()
    return mp


def test_worked_block():
    """amax 7 = 1.75 * 2^2: scale 2^0. Ties go to the even code."""
    x = torch.zeros(1, 32)
    row = [7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, -5.1, 6.9, -0.0, 0.2, 4.9]
    x[0, :len(row)] = torch.tensor(row)
    q, s = mx.quantize(x)
    assert s.tolist() == [[127]]
    want = [6, 0, 1, 1, 2, 2, 4, 4, -0.5, -6, 6, 0, 0, 4]
    assert mx.values(q, s, 32)[0, :len(row)].tolist() == want
    assert q[0, 0].item() == 0x07 and q[0, 5].item() == 0x87   # 7 -> code 7, 0.25 -> 0; 6.9 -> 7, -0.0 -> 8


def test_scale_range():
    x = torch.zeros(5, 32)
    x[1, 0], x[2, 0], x[3, 0], x[4, 0] = 2.0 ** -149, 2.0 ** 127, float("inf"), float("nan")
    assert mx.quantize(x)[1][:, 0].tolist() == [0, 0, 252, 255, 255]


def test_half_the_grid_is_reached():
    """Quantising the values of random codes whose blocks hold a 4 or a 6 gives them back."""
    g = torch.Generator()
    g.manual_seed(1)
    q, s = mx.random_held(g, 40, 100)
    v = mx.values(q, s, 100)
    v[:, ::32] = 4 * torch.exp2(s.double() - 127)
    q2, s2 = mx.quantize(v.float())
    assert torch.equal(s, s2) and torch.equal(mx.values(q2, s2, 100), v)


def quantize(mp, **kw):
    a = dict(h=None, M=4, K=64, type=0, X=P, ldx=64, Q=P, ldq=32, S=P, lds=16, QT=P, ldqt=16, ST=P, ldst=16)
    a.update(kw)
    return mp.mpgemm_quantize_mxfp4(*a.values())


def dequantize(mp, **kw):
    a = dict(h=None, M=4, K=64, Q=P, ldq=32, S=P, lds=16, type=0, Y=P, ldy=64)
    a.update(kw)
    return mp.mpgemm_dequantize_mxfp4(*a.values())


def gemm(mp, **kw):
    a = dict(h=None, M=4, N=8, K=64, A=P, lda=32, SA=P, ldsa=16, B=P, ldb=32, SB=P, ldsb=16, bias=None, type=1, C=P,
             ldc=8, workspace=None, workspace_bytes=0)
    a.update(kw)
    return mp.mpgemm_run_mxfp4(*a.values())


def dyn(mp, **kw):
    a = dict(h=None, M=4, N=8, K=64, type=1, X=P, ldx=64, W=P, ldw=32, SW=P, ldsw=16, bias=None, Y=P, ldy=8,
             workspace=None, workspace_bytes=0)
    a.update(kw)
    return mp.mpgemm_run_mxfp4_dyn(*a.values())


def backward(mp, **kw):
    a = dict(h=None, M=4, N=64, K=8, type=1, dY=P, lddy=64, WT=P, ldwt=32, SWT=P, ldswt=16, XT=P, ldxt=16, SXT=P,
             ldsxt=16, dX=P, lddx=8, dW=P, lddw=8, workspace=None, workspace_bytes=0)
    a.update(kw)
    return mp.mpgemm_run_mxfp4_backward(*a.values())


def newton(mp, **kw):
    a = dict(h=None, batch=2, M=4, N=8, type=1, G=P, ldg=8, strideg=32, steps=5, coeffs=(1., 2., 3.), eps=0.,
             Y=P, ldy=8, stridey=32, workspace=None, workspace_bytes=0)
    a.update(kw)
    return mp.mpgemm_run_newton_schulz(*a.values())


BIG = 1 << 24
CASES = [
    (quantize, dict(M=-1), INVALID), (quantize, dict(K=-1), INVALID), (quantize, dict(type=3), INVALID),
    (quantize, dict(type=-1), INVALID), (quantize, dict(X=None), INVALID), (quantize, dict(ldx=63), INVALID),
    (quantize, dict(ldq=16), INVALID), (quantize, dict(S=None), INVALID), (quantize, dict(Q=None), INVALID),
    (quantize, dict(Q=None, S=None, QT=None, ST=None), INVALID), (quantize, dict(ldst=0), INVALID),
    (quantize, dict(Q=P + 8), UNSUPPORTED), (quantize, dict(S=P + 1), UNSUPPORTED), (quantize, dict(ldq=40), UNSUPPORTED),
    (quantize, dict(lds=18), UNSUPPORTED), (quantize, dict(ldqt=24), UNSUPPORTED), (quantize, dict(X=P + 1), UNSUPPORTED),
    (quantize, dict(X=P + 2, type=2), UNSUPPORTED), (quantize, dict(K=BIG), UNSUPPORTED), (quantize, dict(M=BIG), UNSUPPORTED),
    (quantize, dict(ldq=1 << 23), UNSUPPORTED), (quantize, dict(ldx=1 << 62), UNSUPPORTED),
    (quantize, {}, INVALID),   # the handle
    (dequantize, dict(M=-1), INVALID), (dequantize, dict(type=9), INVALID), (dequantize, dict(Q=None), INVALID),
    (dequantize, dict(Y=None), INVALID), (dequantize, dict(ldy=63), INVALID), (dequantize, dict(lds=1), INVALID),
    (dequantize, dict(Y=P + 1), UNSUPPORTED), (dequantize, dict(Q=P + 4), UNSUPPORTED), (dequantize, dict(K=BIG), UNSUPPORTED),
    (dequantize, {}, INVALID),
    (gemm, dict(M=-1), INVALID), (gemm, dict(N=-1), INVALID), (gemm, dict(K=-1), INVALID), (gemm, dict(type=3), INVALID),
    (gemm, dict(A=None), INVALID), (gemm, dict(SB=None), INVALID), (gemm, dict(C=None), INVALID), (gemm, dict(ldc=7), INVALID),
    (gemm, dict(lda=16), INVALID), (gemm, dict(ldsb=1), INVALID), (gemm, dict(B=P + 2), UNSUPPORTED),
    (gemm, dict(ldb=33), UNSUPPORTED), (gemm, dict(ldsa=17), UNSUPPORTED), (gemm, dict(bias=P + 1), UNSUPPORTED),
    (gemm, dict(bias=P + 2, type=2), UNSUPPORTED), (gemm, dict(C=P + 1), UNSUPPORTED), (gemm, dict(K=BIG), UNSUPPORTED),
    (gemm, dict(M=BIG), UNSUPPORTED), (gemm, {}, INVALID),
    (dyn, dict(M=-1), INVALID), (dyn, dict(type=3), INVALID), (dyn, dict(X=None), INVALID), (dyn, dict(ldx=63), INVALID),
    (dyn, dict(W=None), INVALID), (dyn, dict(ldw=16), INVALID), (dyn, dict(Y=None), INVALID), (dyn, dict(ldy=7), INVALID),
    (dyn, dict(X=P + 1), UNSUPPORTED), (dyn, dict(SW=P + 8), UNSUPPORTED), (dyn, dict(bias=P + 1), UNSUPPORTED),
    (dyn, dict(N=BIG), UNSUPPORTED), (dyn, {}, INVALID),
    (backward, dict(M=-1), INVALID), (backward, dict(type=3), INVALID), (backward, dict(dY=None), INVALID),
    (backward, dict(dX=None, dW=None), INVALID), (backward, dict(WT=None), INVALID), (backward, dict(XT=None), INVALID),
    (backward, dict(lddx=7), INVALID), (backward, dict(lddw=7), INVALID), (backward, dict(lddy=63), INVALID),
    (backward, dict(ldwt=16), INVALID), (backward, dict(dW=P + 2), UNSUPPORTED), (backward, dict(SXT=P + 4), UNSUPPORTED),
    (backward, dict(M=BIG), UNSUPPORTED), (backward, {}, INVALID),
    (newton, dict(batch=-1), INVALID), (newton, dict(M=-1), INVALID), (newton, dict(type=3), INVALID),
    (newton, dict(steps=-1), INVALID), (newton, dict(eps=-1.0), INVALID), (newton, dict(eps=float("nan")), INVALID),
    (newton, dict(coeffs=None), INVALID), (newton, dict(G=None), INVALID), (newton, dict(Y=None), INVALID),
    (newton, dict(ldg=7), INVALID), (newton, dict(ldy=7), INVALID), (newton, dict(stridey=31), INVALID),
    (newton, dict(type=2), UNSUPPORTED), (newton, dict(steps=101), UNSUPPORTED), (newton, dict(G=P + 1), UNSUPPORTED),
    (newton, dict(M=1 << 17), UNSUPPORTED), (newton, dict(batch=1 << 16), UNSUPPORTED), (newton, {}, INVALID),
]


@pytest.mark.parametrize("call,args,want", CASES, ids=[f"{c.__name__}-{'-'.join(a)or'handle'}-{i}" for i, (c, a, _) in enumerate(CASES)])
def test_refusals(mp, call, args, want):
    assert call(mp, **args) == want


def test_no_ops(mp):
    assert quantize(mp, M=0) == 0 and quantize(mp, K=0) == 0
    assert dequantize(mp, M=0) == 0 and dequantize(mp, K=0) == 0
    assert gemm(mp, M=0) == 0 and gemm(mp, N=0) == 0
    assert dyn(mp, M=0) == 0 and dyn(mp, N=0) == 0
    assert backward(mp, K=0) == 0 and backward(mp, M=0, N=0) == 0
    assert newton(mp, batch=0) == 0 and newton(mp, M=0) == 0 and newton(mp, N=0) == 0


def test_workspaces(mp):
    assert mp.mpgemm_run_mxfp4_workspace(-1, 4, 4) == -1
    assert mp.mpgemm_run_mxfp4_workspace(4, 4, BIG) == -1
    assert mp.mpgemm_run_mxfp4_workspace(0, 4, 4) == 0
    assert mp.mpgemm_run_mxfp4_workspace(4096, 4096, 4096) == 0
    assert mp.mpgemm_run_mxfp4_dyn_workspace(1, 4096, 4096) == 0
    # codes and scales of X
    assert mp.mpgemm_run_mxfp4_dyn_workspace(2048, 4096, 4096) >= 2048 * 4096 * 17 // 32
    assert mp.mpgemm_run_mxfp4_backward_workspace(4096, 4096, 4096) >= 2 * 4096 * 4096 * 17 // 32
    assert mp.mpgemm_run_mxfp4_backward_workspace(0, 64, 64) == 0
    assert mp.mpgemm_run_newton_schulz_workspace(-1, 4, 4) == -1
    assert mp.mpgemm_run_newton_schulz_workspace(0, 4, 4) == 0
    # a long batch is worked off in parts
    assert mp.mpgemm_run_newton_schulz_workspace(60000, 512, 512) <= 5 << 30


def test_torch_layer_refusals(mp):
    """Host tensors, wrong types and shapes raise before anything is launched."""
    x = torch.zeros(4, 64)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mp.quantize_mxfp4(x)
    with pytest.raises(TypeError):
        mp.quantize_mxfp4(x.double())
    with pytest.raises(TypeError):
        mp.quantize_mxfp4_both(x.to(torch.int8))
    with pytest.raises(ValueError):
        mp.gemm_mxfp4_dyn(x, q, s)
    with pytest.raises(ValueError):
        mp.gemm_mxfp4(q, s, q, s, 64)
    with pytest.raises(TypeError):
        mp.gemm_mxfp4(q, s, q, s, 64, dtype=torch.float64)
    with pytest.raises(ValueError):
        mp.dequantize_mxfp4(q, s, 64)
    with pytest.raises(ValueError):
        mp.gemm_mxfp4_backward(x, q, s, q, s)
    with pytest.raises(TypeError):
        mp.newton_schulz(x)
    with pytest.raises(ValueError):
        mp.newton_schulz(x.half()[0])
    with pytest.raises(ValueError):
        mp.newton_schulz(x.half(), coeffs=(1.0, 2.0))
    with pytest.raises(ValueError):
        mp.newton_schulz(x.half())
