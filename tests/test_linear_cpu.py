"""Refusals and workspace sizes of the 8-bit integer and gated calls, without a GPU: argument errors come before any
device work (the handle is checked last, so a NULL handle reaches every check), and calls that take tensors refuse before they touch a device."""
import os

import pytest
import torch

A, B, C, S, D = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000   # never dereferenced


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    if not os.path.exists(mp.lib_path) or not os.path.exists(mp.calls_path):
        from precision_dense_gemm_tiled_amd import build
        build.build()
    return mp


@pytest.mark.parametrize("args,expect", [
    ((-1, 4, 0, A, 4, B, 16, S), 1), ((4, 4, 7, A, 4, B, 16, S), 1),
    ((0, 4, 0, 0, 4, 0, 16, 0), 0), ((4, 0, 0, 0, 4, 0, 16, 0), 0),
    ((4, 4, 0, 0, 4, B, 16, S), 1), ((4, 4, 0, A, 3, B, 16, S), 1), ((4, 4, 0, A, 4, B, 3, S), 1), ((4, 4, 0, A, 4, B, 16, 0), 1),
    ((4, 4, 0, A + 1, 4, B, 16, S), 2), ((4, 4, 2, A + 2, 4, B, 16, S), 2), ((4, 4, 0, A, 4, B, 16, S + 2), 2),
    (((1 << 24) + 1, 4, 0, A, 4, B, 16, S), 2),
    ((4, 4, 0, A + 2, 4, B + 1, 5, S), 1),   # (fine: the NULL handle is left)
])
def test_quantize_refusals(mp, args, expect):
    assert mp.mpgemm_quantize_i8(None, *args) == expect
    M, K, t, X, ldx, Q, ldq, Sc = args
    if Q == B and X == A:
        assert mp.mpgemm_dequantize_i8(None, M, K, Q, ldq, Sc, t, X, ldx) == expect


W8 = dict(M=4, N=6, K=32, A=A, lda=32, SA=S, B=B, ldb=32, SB=S, bias=None, type=0, C=C, ldc=6)


@pytest.mark.parametrize("change,expect", [
    ({}, 1), (dict(M=-1), 1), (dict(M=0, A=0, C=0), 0), (dict(N=0), 0), (dict(type=3), 1),
    (dict(A=0), 1), (dict(SA=0), 1), (dict(B=0), 1), (dict(SB=0), 1), (dict(C=0), 1), (dict(lda=31), 1), (dict(ldb=31), 1), (dict(ldc=5), 1),
    (dict(SA=S + 1), 2), (dict(SB=S + 2), 2), (dict(C=C + 1), 2), (dict(type=2, C=C + 2), 2), (dict(bias=D + 1), 2), (dict(type=2, bias=D + 2), 2),
    (dict(K=131072, lda=131072, ldb=131072), 2), (dict(M=(1 << 24) + 1), 2),
    (dict(A=A + 1, lda=33, B=B + 3, ldb=35), 1),   # (any alignment: the NULL handle is left)
    (dict(K=0, A=0, B=0, SA=0, SB=0), 1),
])
def test_product_refusals(mp, change, expect):
    p = {**W8, **change}
    assert mp.mpgemm_run_w8a8(None, *p.values()) == expect
    # the dynamic call: X takes the place of the codes (fp16: its row stride counts elements)
    x = 0 if p["A"] == 0 else A
    if "SA" not in change and not (p["A"] and p["A"] != A):
        assert mp.mpgemm_run_w8a8_dyn(None, p["M"], p["N"], p["K"], p["type"], x, p["lda"], p["B"], p["ldb"], p["SB"], p["bias"], p["C"], p["ldc"]) == expect
    if "bias" not in change:
        for act, e in ((0, expect), (2, expect), (3, 1), (-1, 1)):
            got = mp.mpgemm_run_gated_w8a8(None, p["M"], p["N"], p["K"], act, p["A"], p["lda"], p["SA"], p["B"], p["ldb"], p["SB"], p["B"], p["ldb"],
                                           p["SB"], p["type"], p["C"], p["ldc"])
            assert got == e


GATED = dict(M=4, N=6, K=32, type=1, act=0, X=A, ldx=32, Wg=B, ldwg=32, Wu=B, ldwu=40, H=C, ldh=6, G=None, ldg=0, U=None, ldu=0)


@pytest.mark.parametrize("change,expect", [
    ({}, 1), (dict(M=-2), 1), (dict(M=0), 0), (dict(N=0), 0), (dict(type=2), 1), (dict(act=3), 1), (dict(X=0), 1), (dict(Wg=0), 1), (dict(Wu=0), 1),
    (dict(H=0), 1), (dict(ldx=31), 1), (dict(ldwg=31), 1), (dict(ldwu=31), 1), (dict(ldh=5), 1), (dict(G=D, ldg=6), 1), (dict(U=D, ldu=6), 1),
    (dict(G=D, ldg=5, U=D, ldu=6), 1), (dict(G=D, ldg=6, U=D + 1, ldu=6), 2), (dict(X=A + 1), 2), (dict(H=C + 1), 2),
    (dict(K=1 << 22, ldx=1 << 22, ldwg=1 << 22, ldwu=1 << 22), 2), (dict(K=0, X=0, Wg=0, Wu=0), 1),
])
def test_gated_refusals(mp, change, expect):
    assert mp.mpgemm_run_gated(None, *{**GATED, **change}.values()) == expect


BACK = dict(M=4, N=6, K=32, type=0, act=1, dH=A, lddh=6, X=A, ldx=32, Wg=B, ldwg=32, Wu=B, ldwu=40, G=D, ldg=6, U=D, ldu=6, dX=C, lddx=32,
            dWg=C, lddwg=32, dWu=C, lddwu=33)


@pytest.mark.parametrize("change,expect", [
    ({}, 1), (dict(K=-1), 1), (dict(type=2), 1), (dict(act=5), 1), (dict(dX=None, dWg=None, dWu=None), 0), (dict(K=0), 0), (dict(dH=0), 1), (dict(G=0), 1),
    (dict(U=0), 1), (dict(X=0), 1), (dict(Wg=0), 1), (dict(lddh=5), 1), (dict(lddx=31), 1), (dict(lddwg=31), 1), (dict(lddwu=31), 1), (dict(ldg=5), 1),
    (dict(dX=C + 1), 2), (dict(dWu=C + 1), 2), (dict(dH=A + 1), 2), (dict(N=1 << 21, lddh=1 << 21, ldg=1 << 21, ldu=1 << 21), 2),
    (dict(dX=None, Wg=0, Wu=0), 1), (dict(dWg=None, dWu=None, X=0), 1),
])
def test_backward_refusals(mp, change, expect):
    assert mp.mpgemm_run_gated_backward(None, *{**BACK, **change}.values()) == expect


def test_workspaces(mp):
    cus = 256
    assert mp.mpgemm_run_w8a8_workspace(4, 4096, 4096, 0, cus) == 0
    assert mp.mpgemm_run_w8a8_workspace(300, 500, 112, 1, cus) == 0
    assert mp.mpgemm_run_w8a8_workspace(300, 500, 100, 1, cus) >= 300 * 112         # k ends inside 16 bytes
    assert mp.mpgemm_run_w8a8_workspace(300, 500, 100, 0, cus) >= 300 * 112 + 500 * 112
    assert mp.mpgemm_run_w8a8_dyn_workspace(1, 4096, 4096, 0, cus) == 0            # quantised by the product
    assert mp.mpgemm_run_w8a8_dyn_workspace(300, 500, 100, 1, cus) >= 300 * 112 + 1200
    assert mp.mpgemm_run_gated_workspace(4096, 1024, 512, 1, cus) == 0
    assert mp.mpgemm_run_gated_workspace(300, 100, 50, 0, cus) >= (300 + 200) * 112
    assert mp.mpgemm_run_gated_backward_workspace(300, 100, 64, 1, cus) >= 300 * 2 * 128 * 2
    for f in (mp.mpgemm_run_w8a8_workspace, mp.mpgemm_run_w8a8_dyn_workspace, mp.mpgemm_run_gated_w8a8_workspace, mp.mpgemm_run_gated_w8a8_dyn_workspace):
        assert f(4, 4, 131072, 1, cus) == -1 and f(-1, 4, 4, 1, cus) == -1 and f(4, 4, 4, 1, 0) == -1 and f(0, 4, 4, 1, cus) == 0
    assert mp.mpgemm_run_gated_workspace(4, 4, 1 << 22, 1, cus) == -1
    assert mp.mpgemm_run_gated_backward_workspace(4, 1 << 21, 4, 1, cus) == -1


def host(mp):
    h = lambda r, c: torch.zeros(r, c, dtype=torch.float16)   # noqa: E731
    q, s = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    return {"dyn X": ((4, 64), lambda t: mp.gemm_w8a8_dyn(t, q, s)),
            "gated X": ((4, 64), lambda t: mp.gemm_gated(t, h(8, 64), h(8, 64))),
            "gated backward dH": ((4, 8), lambda t: mp.gemm_gated_backward(t, h(4, 64), h(8, 64), h(8, 64), h(4, 8), h(4, 8))),
            "gated integers X": ((4, 64), lambda t: mp.gemm_gated_w8a8_dyn(t, q, s, q, s))}


@pytest.mark.parametrize("name", ["dyn X", "gated X", "gated backward dH", "gated integers X"])
def test_a_lost_gradient_raises(mp, name):
    shape, call = host(mp)[name]
    make = lambda: torch.zeros(shape, dtype=torch.float16)   # noqa: E731
    with pytest.raises(RuntimeError, match="autograd"):
        call(make().requires_grad_())
    with pytest.raises(ValueError, match="device tensor"):
        call(make())
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
        call(make().requires_grad_())


def test_types_are_refused(mp):
    h = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        mp.gemm_gated(h.float(), h.float(), h.float())
    with pytest.raises(TypeError):
        mp.quantize_i8(h.double())
    with pytest.raises(TypeError):
        mp.gemm_w8a8(h, torch.zeros(4), h, torch.zeros(4))
    with pytest.raises(TypeError):
        mp.gemm_w8a8_dyn(h.to(torch.int8), h.to(torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="act"):
        mp.gemm_gated(h, h, h, act="relu")
