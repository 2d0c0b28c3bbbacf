"""Calls of the 8-bit integer layer and the gated block at the ends of what they take: single rows of great length, held
matrices that are saved and loaded, gates far below zero, gradients that only one weight needs."""
import pytest
import torch

from . import linear_util as lu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    assert torch.cuda.is_available()
    return mp


# One row as long as 2^23 bytes and more: it has no stride, and is taken as it lies (or, not at 16 bytes, from a copy).
@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("M,N,K,need", [(1, 8, 1 << 22, "w"), (1, 1, 1 << 22, "xw"), (66, 1, 1 << 22, "x"), (1, 8, 1 << 24, "w"), (1, 1, 1 << 24, "xw")])
def test_backward_of_one_long_row(mp, M, N, K, need, at):
    dt = torch.bfloat16
    gg = torch.Generator(device="cuda").manual_seed(M + N + K)

    def rows(r):
        big = torch.empty(r * K + 8, device="cuda", dtype=dt)[at:at + r * K].view(r, K)
        return big.copy_(torch.randn(r, K, generator=gg, device="cuda", dtype=dt))

    x, wg, wu = rows(M), rows(N), rows(N)
    dh, g, u = (torch.randn(M, N, generator=gg, device="cuda", dtype=dt) for _ in range(3))
    got = mp.gemm_gated_backward(dh, x if "w" in need else None, wg if "x" in need else None, wu if "x" in need else None, g, u,
                                 need_dx="x" in need, need_dw="w" in need)
    assert [v is None for v in got] == ["x" not in need, "w" not in need, "w" not in need]
    for k in (slice(0, 300), slice(K // 2 - 5, K // 2 + 200), slice(K - 300, K)):
        want = lu.gated_backward(*(v.cpu() for v in (dh, x[:, k], wg[:, k], wu[:, k], g, u)), "silu", dt)
        for y, (w, e) in zip(got, want):
            if y is not None:
                lu.check(y[:, k], w, e)


# Weights brought into integers are kept in a checkpoint: codes and scales save and load, alone and together.
@pytest.mark.parametrize("N,K", [(40, 200), (64, 512), (1, 7), (3, 16)])
def test_held_matrices_are_saved_and_loaded(mp, tmp_path, N, K):
    gg = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(5, K, generator=gg, device="cuda").bfloat16()
    q, s = mp.quantize_i8(torch.randn(N, K, generator=gg, device="cuda"))
    assert q.untyped_storage().data_ptr() != s.untyped_storage().data_ptr()
    assert s.untyped_storage().nbytes() == 4 * N   # (and scales alone keep no codes)
    want = mp.gemm_w8a8_dyn(x, q, s)
    torch.save({"q": q, "s": s}, tmp_path / "held.pt")
    held = torch.load(tmp_path / "held.pt", weights_only=True)
    assert torch.equal(held["q"], q) and torch.equal(held["s"], s)
    assert torch.equal(mp.gemm_w8a8_dyn(x, held["q"], held["s"]), want)
    host = torch.load(tmp_path / "held.pt", weights_only=True, map_location="cpu")
    assert torch.equal(mp.gemm_w8a8_dyn(x, host["q"].cuda(), host["s"].cuda()), want)
