"""Codes and scales after ordinary tensor handling, which drops the padding of the scale rows."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

pytestmark = pytest.mark.gpu

COPIES = {"clone": lambda t: t.clone(), "contiguous": lambda t: t.contiguous(), "host and back": lambda t: t.cpu().cuda(),
          "rows of a larger one": lambda t: torch.cat([t[:1], t])[1:], "odd offset": lambda t: torch.cat([t, t], 1)[:, t.shape[1]:]}


@pytest.mark.parametrize("copy", list(COPIES))
@pytest.mark.parametrize("M,N,K", [(1, 100, 520), (16, 100, 2100), (64, 130, 520), (100, 1, 520), (333, 200, 70), (2, 3, 1)])
def test_copied_scales(M, N, K, copy):
    g = torch.Generator()
    g.manual_seed(M + N + K)
    x, w, dy = (torch.randn(r, c, generator=g).bfloat16().cuda() for r, c in ((M, K), (N, K), (M, N)))
    xq, xs, xtq, xts = mp.quantize_mxfp4_both(x)
    wq, ws, wtq, wts = mp.quantize_mxfp4_both(w)
    c = COPIES[copy]
    assert torch.equal(mp.dequantize_mxfp4(wq, c(ws), K), mp.dequantize_mxfp4(wq, ws, K))
    assert torch.equal(mp.gemm_mxfp4(xq, c(xs), wq, c(ws), K), mp.gemm_mxfp4(xq, xs, wq, ws, K))
    assert torch.equal(mp.gemm_mxfp4_dyn(x, wq, c(ws)), mp.gemm_mxfp4_dyn(x, wq, ws))
    for a, b in zip(mp.gemm_mxfp4_backward(dy, wtq, c(wts), xtq, c(xts)), mp.gemm_mxfp4_backward(dy, wtq, wts, xtq, xts)):
        assert torch.equal(a, b)


def test_copied_scales_in_a_graph_and_on_a_stream():
    g = torch.Generator()
    g.manual_seed(1)
    x, w = torch.randn(70, 520, generator=g).half().cuda(), torch.randn(90, 520, generator=g).half().cuda()
    q, s = mp.quantize_mxfp4(w)
    flat = s.clone()
    assert flat.stride(0) == 17
    want = mp.gemm_mxfp4_dyn(x, q, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mp.gemm_mxfp4_dyn(x, q, flat)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        q2, s2 = mp.quantize_mxfp4(w)   # eager work between the replays
        assert torch.equal(mp.gemm_mxfp4_dyn(x, q2, s2.clone()), want)
    other = mp.gemm_mxfp4_dyn(x, q, flat, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(other, want)
