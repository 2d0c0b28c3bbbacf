"""The scratch of the 8-bit integer and gated calls, without a GPU: a call takes exactly the bytes that its _workspace call
names for the operands it is given, and refuses fewer. A stand-in handle of a device that no machine has lets a call come as
far as its check of the workspace and no further: what passes ends with MPGEMM_ERR_HIP before any kernel."""
import ctypes
import os
import random

import pytest

ARG, HIP = 1, 4
CUS = 256


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    if not os.path.exists(mp.lib_path):
        from precision_dense_gemm_tiled_amd import build
        build.build()
    return mp


@pytest.fixture(scope="module")
def handle():
    buf = (ctypes.c_int * 64)(1000, CUS)   # (the context's first members: device, compute units)
    yield ctypes.addressof(buf)
    del buf


P = 1 << 20   # a 16-byte aligned address, never dereferenced


class Rows:
    """Where a matrix lies: its address and row stride (elements of `size` bytes)."""
    def __init__(self, rows, cols, size, at=P, ld=None):
        self.rows, self.size, self.at, self.ld = rows, size, at, cols if ld is None else ld

    def aligned(self):
        return self.at % 16 == 0 and (self.rows <= 1 or (self.ld * self.size % 16 == 0 and self.ld * self.size < 1 << 23))


def some_rows(rng, rows, cols, size):
    at = P + size * rng.choice([0, 0, 0, 1, 8, 5])
    ld = cols + rng.choice([0, 0, 1, 3, -cols % 16, -cols % 16 + 16, (1 << 23) - cols if cols < 1 << 23 else 0])
    return Rows(rows, cols, size, at, ld)


def backward(mp, h, M, N, K, X, Wg, Wu, need_dx=True, need_dw=True):
    al = all(o.aligned() for o in ([X] if need_dw else []) + ([Wg, Wu] if need_dx else [])) and (not need_dx or N <= 1 or Wg.ld == Wu.ld)
    n = mp.mpgemm_run_gated_backward_workspace(M, N, K, al, CUS)
    take = lambda b: mp.mpgemm_run_gated_backward(h, M, N, K, 0, 0, P, N, X.at, X.ld, Wg.at, Wg.ld, Wu.at, Wu.ld, P, N, P, N,   # noqa: E731
                                                  P if need_dx else None, K, P if need_dw else None, K, P if need_dw else None, K, P, b)
    return n, take, al and need_dx and need_dw


# One row as long as 2^23 bytes and more: it has no stride that could be too long.
@pytest.mark.parametrize("M,N,K,dx,dw", [(1, 8, 1 << 22, False, True), (1, 1, 1 << 22, True, True), (66, 1, 1 << 22, True, False),
                                         (1, 8, 1 << 24, False, True), (1, 1, 1 << 24, True, True), (1, 3, (1 << 22) - 8, True, True)])
def test_backward_of_one_long_row(mp, handle, M, N, K, dx, dw):
    n, take, _ = backward(mp, handle, M, N, K, Rows(M, K, 2), Rows(N, K, 2), Rows(N, K, 2), dx, dw)
    assert take(n) == HIP
    assert take(n - 1) == ARG


@pytest.mark.parametrize("seed", range(40))
def test_the_scratch_that_is_named_is_what_a_call_takes(mp, handle, seed):
    rng = random.Random(seed)
    size = lambda *more: rng.choice([1, 2, 3, 16, 31, 32, 33, 64, 100, 513, 2048, *more])   # noqa: E731
    for _ in range(20):
        M, N, K = size(), size(), size(777, 4096, 8200)
        # in 16 bits
        X, Wg, Wu = (some_rows(rng, r, K, 2) for r in (M, N, N))
        al = X.aligned() and Wg.aligned() and Wu.aligned()
        n = mp.mpgemm_run_gated_workspace(M, N, K, al, CUS)
        assert mp.mpgemm_run_gated(handle, M, N, K, 1, 0, X.at, X.ld, Wg.at, Wg.ld, Wu.at, Wu.ld, P, N, None, 0, None, 0, P, n) == HIP
        for need in ((True, True), (True, False), (False, True)):
            n, take, exact = backward(mp, handle, M, N, K, X, Wg, Wu, *need)
            assert take(n) == HIP
            assert not exact or take(n - 1) == ARG
        # on integers
        t = rng.choice([0, 1, 2])
        A, B, B2 = (some_rows(rng, r, K, 1) for r in (M, N, N))
        al, albs = A.aligned(), B.aligned() and B2.aligned()
        n = mp.mpgemm_run_w8a8_workspace(M, N, K, al and B.aligned(), CUS)
        assert mp.mpgemm_run_w8a8(handle, M, N, K, A.at, A.ld, P, B.at, B.ld, P, None, t, P, N, P, n) == HIP
        n = mp.mpgemm_run_w8a8_dyn_workspace(M, N, K, B.aligned(), CUS)
        assert mp.mpgemm_run_w8a8_dyn(handle, M, N, K, t, P, K + 1, B.at, B.ld, P, None, P, N, P, n) == HIP
        assert n == 0 or mp.mpgemm_run_w8a8_dyn(handle, M, N, K, t, P, K + 1, B.at, B.ld, P, None, P, N, P, n - 1) == ARG or not B.aligned()
        n = mp.mpgemm_run_gated_w8a8_workspace(M, N, K, al and albs, CUS)
        assert mp.mpgemm_run_gated_w8a8(handle, M, N, K, 1, A.at, A.ld, P, B.at, B.ld, P, B2.at, B2.ld, P, t, P, N, P, n) == HIP
        n = mp.mpgemm_run_gated_w8a8_dyn_workspace(M, N, K, albs, CUS)
        assert mp.mpgemm_run_gated_w8a8_dyn(handle, M, N, K, t, 2, P, K, B.at, B.ld, P, B2.at, B2.ld, P, P, N, P, n) == HIP
