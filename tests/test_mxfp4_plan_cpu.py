"""Which kernel takes a product of few rows, seen from the scratch: a tile product of few tiles and a long K keeps
partial sums in it, the skinny kernel none."""
import os

import pytest


@pytest.fixture(scope="module")
def need():
    import precision_dense_gemm_tiled_amd as mp
    if not os.path.exists(mp.lib_path):
        from precision_dense_gemm_tiled_amd import build
        build.build()
    return mp.mpgemm_run_mxfp4_workspace


@pytest.mark.parametrize("M,N,K", [(33, 2048, 16384), (64, 256, 8192), (64, 4096, 12288), (48, 1024, 12288), (32, 2048, 16384)])
def test_long_rows_go_through_tiles(need, M, N, K):
    assert need(M, N, K) > 0


@pytest.mark.parametrize("M,N,K", [(1, 4096, 1 << 20), (4, 2048, 16384), (16, 4096, 16384), (17, 2048, 16384), (32, 1024, 12288), (64, 4096, 6144),
                                   (48, 8192, 8192), (64, 4096, 1024)])
def test_others_do_not(need, M, N, K):
    assert need(M, N, K) == 0
