"""MXFP4 and Newton-Schulz at the sizes where their launch plans change, against 64 bits."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

from . import mx_util as mx

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def product(A, B, K):
    a, b = mx.values(*A, K), mx.values(*B, K)
    return a @ b.t(), a.abs() @ b.abs().t()


# few rows of 8192 columns and more, 32 per workgroup (33 and 64 rows: at 8192, beyond it tiles); K in one group of 16
# blocks, several, and a last group of one block; rows of each block of 16
@pytest.mark.parametrize("M", [1, 3, 16, 17, 33, 64])
@pytest.mark.parametrize("N,K", [(8192, 512), (8200, 1056), (8209, 5000)])
def test_wide_skinny(M, N, K):
    g = gen(M + N + K)
    A, B = mx.random_held(g, M, K), mx.random_held(g, N, K)
    B[1][:, -1] = 126
    bias = torch.randn(N, generator=g).bfloat16()
    y, t = product(A, B, K)
    y, t = y + bias.double(), t + bias.double().abs()
    got = mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), K, bias=bias.cuda(), dtype=torch.bfloat16)
    mx.check(got, y, mx.gemm_tol(y, t, (K + 31) // 32, torch.bfloat16))


# few rows of many columns, on both sides of the sizes from which tiles take them
@pytest.mark.parametrize("M,N,K", [(64, 8193, 300), (33, 9000, 2100), (32, 10239, 520), (32, 10240, 520), (17, 12000, 1100),
                                   (16, 24575, 264), (16, 24576, 264), (5, 24577, 1030), (4, 24600, 520), (1, 30000, 1000)])
@pytest.mark.parametrize("name", ["f16", "f32"])
def test_few_rows_of_many_columns(M, N, K, name):
    g = gen(M + N + K)
    dtype = {"f16": torch.float16, "f32": torch.float32}[name]
    x = (torch.randn(M, K, generator=g) * 0.1).to(dtype)
    W = mx.random_held(g, N, K, spread=1)
    w = mx.on_gpu(W)
    bias = torch.randn(N, generator=g).to(dtype)
    out = mp.gemm_mxfp4_dyn(x.cuda(), *w, bias=bias.cuda())
    X = mx.quantize(x)
    y, t = product(X, W, K)
    tol = mx.gemm_tol(y + bias.double(), t + bias.double().abs(), (K + 31) // 32 + 1, dtype)
    mx.check(out, y + bias.double(), tol)
    assert torch.equal(mp.gemm_mxfp4(*mx.on_gpu(X), *w, K, bias=bias.cuda(), dtype=dtype), out)


# activations quantised by the product itself: one piece of 8 per thread, four, and the most rows that still are;
# rows that are not 16-byte aligned or whose length is not a multiple of 8
@pytest.mark.parametrize("M,K,pad", [(1, 8, 0), (1, 4096, 0), (2, 4096, 0), (1, 16384, 0), (16, 1000, 0), (16, 1024, 8),
                                     (4, 4095, 1), (4, 4096, 3), (5, 2044, 4)])
@pytest.mark.parametrize("name", ["f16", "f32"])
def test_fused_quantisation(M, K, pad, name):
    g = gen(M + K + pad)
    dt = mx.TYPES[name]
    x = (torch.randn(M, K + pad, generator=g) * torch.exp2(torch.randint(-8, 5, (M, K + pad), generator=g).float())).to(dt)
    W = mx.random_held(g, 100, K, spread=1)
    xg = x.cuda()[:, pad:]
    assert mp.mpgemm_run_mxfp4_dyn_workspace(M, 100, K) == 0
    got = mp.gemm_mxfp4_dyn(xg, *mx.on_gpu(W))
    y, t = product(mx.quantize(x[:, pad:]), W, K)
    mx.check(got, y, mx.gemm_tol(y, t, (K + 31) // 32, dt))
    q, s = mp.quantize_mxfp4(xg)
    assert torch.equal(got, mp.gemm_mxfp4(q, s, *mx.on_gpu(W), K, dtype=dt))


# quantisation with one row per thread and with four; pieces past the row, few and many
@pytest.mark.parametrize("M,K", [(4096, 1024), (3001, 1500), (65, 9000), (20000, 40), (1, 20000)])
@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_long_quantisation(M, K, name):
    g = gen(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-8, 5, (M, 1), generator=g).float())).to(mx.TYPES[name])
    q, s = mp.quantize_mxfp4(x.cuda())
    wq, ws = mx.quantize(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)
    y = mp.dequantize_mxfp4(q, s, K, mx.TYPES[name])
    assert torch.equal(y.cpu().double(), mx.values(wq, ws, K))


# both gradients in one grid of 64, 128 and 256 tiles, with ragged edges; K of one stage and of an odd number
@pytest.mark.parametrize("M,N,K", [(100, 90, 200), (300, 257, 1000), (2100, 1100, 1300), (1500, 2050, 2000), (4100, 4000, 2300)])
def test_backward_pairs(M, N, K):
    g = gen(M + N + K)
    dy = (torch.randn(M, N, generator=g) * torch.exp2(torch.randint(-6, 3, (M, 1), generator=g).float())).bfloat16()
    WT, XT = mx.random_held(g, K, N, spread=1), mx.random_held(g, K, M, spread=1)
    wt, xt = mx.on_gpu(WT), mx.on_gpu(XT)
    dx, dw = mp.gemm_mxfp4_backward(dy.cuda(), *wt, *xt)
    rows = slice(0, M, max(1, M // 200))
    y, t = product(mx.quantize(dy[rows]), WT, N)
    mx.check(dx[rows], y, mx.gemm_tol(y, t, (N + 31) // 32, torch.bfloat16))
    cols = slice(0, N, max(1, N // 200))
    y, t = product(mx.quantize(dy.t()[cols]), XT, M)
    mx.check(dw[cols], y, mx.gemm_tol(y, t, (M + 31) // 32, torch.float32))
    # every output, from the single products of the same quantised gradient
    q, s, qt, st = mp.quantize_mxfp4_both(dy.cuda())
    assert torch.equal(dx, mp.gemm_mxfp4(q, s, *wt, N, dtype=torch.bfloat16))
    assert torch.equal(dw, mp.gemm_mxfp4(qt, st, *xt, M))


# tiles of 128 and 256 on one and on several workgroups per CU, ragged, in products and pairs
@pytest.mark.parametrize("M,N,K", [(2000, 4000, 1000), (2048, 4097, 296), (4090, 2000, 72), (1900, 1100, 2600)])
@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_large_tiles(M, N, K, name):
    g = gen(M + N + K)
    A, B = mx.random_held(g, M, K, spread=1), mx.random_held(g, N, K, spread=1)
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[name]
    out = mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), K, dtype=dtype)
    rows = torch.cat([torch.arange(0, M, max(1, M // 100)), torch.arange(M - 3, M)])
    y, t = product((A[0][rows], A[1][rows]), B, K)
    mx.check(out[rows.cuda()], y, mx.gemm_tol(y, t, (K + 31) // 32, dtype))
    whole = mp.gemm_mxfp4(*mx.on_gpu((A[0][:65], A[1][:65])), *mx.on_gpu(B), K, dtype=dtype)   # smaller tiles
    assert torch.equal(out[:65], whole) or K > 2048   # (few rows and a long K: the sum is split)


@pytest.mark.parametrize("M,N,K", [(1500, 1000, 1000), (1000, 1000, 4000), (2000, 2100, 1900)])
def test_backward_pairs_of_large_tiles(M, N, K):
    test_backward_pairs(M, N, K)


def test_a_held_pair_shares_its_allocation():
    q, s, qt, st = mp.quantize_mxfp4_both(torch.ones(40, 70, device="cuda"))
    assert q.untyped_storage().data_ptr() == s.untyped_storage().data_ptr()
    assert q.untyped_storage().data_ptr() != qt.untyped_storage().data_ptr()
    assert q.stride() == (48, 1) and s.shape == (40, 3) and s.stride() == (16, 1) and st.shape == (70, 2)
    assert torch.equal(q.clone(), q) and torch.equal(s.contiguous(), s)


def grads(g, B, M, N, dtype, noise=1.0, rank=16):
    r = min(M, N, rank)
    low = torch.randn(B, M, r, generator=g) @ torch.randn(B, r, N, generator=g)
    return (1e-3 * (low + noise * torch.randn(B, M, N, generator=g))).to(dtype)


# 128 x 128 tiles on at most one and on more than one workgroup per CU, single steps and groups
@pytest.mark.parametrize("B,M,N", [(13, 512, 512), (27, 512, 400), (27, 300, 512), (2, 1500, 1030), (1, 2100, 700)])
def test_newton_schulz_large_tiles(B, M, N):
    g = gen(B + M + N)
    x = grads(g, B, M, N, torch.bfloat16)
    got = mp.newton_schulz(x.cuda())
    for b in (0, B - 1):
        want = mx.newton_schulz(x[b])
        off, norm = torch.linalg.vector_norm(got[b].double().cpu() - want), torch.linalg.vector_norm(want)
        # half a step of the output for its rounding, an eighth of one for the iteration
        assert off <= mx.half_step(torch.bfloat16) * 1.125 * norm
        assert torch.equal(mp.newton_schulz(x[b].cuda()), got[b])


# sides up to 128, where one workgroup takes all steps of a group, and beyond; the long side short, one slice of it,
# several with a ragged last one, and as many as there are
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("B,M,N", [(2, 64, 512), (1, 64, 4096), (5, 50, 2900), (2, 100, 1024), (1, 128, 5000), (4, 3000, 127),
                                   (1, 20, 20000), (1, 129, 1100), (3, 192, 768), (1, 192, 2500), (2, 256, 4096), (1, 700, 2900)])
def test_newton_schulz_long_and_narrow(B, M, N, name):
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16}[name]
    g = gen(B + M + N)
    x = grads(g, B, M, N, dtype)
    got = mp.newton_schulz(x.cuda())
    for b in range(B):
        want = mx.newton_schulz(x[b])
        off, norm = torch.linalg.vector_norm(got[b].double().cpu() - want), torch.linalg.vector_norm(want)
        assert off <= mx.half_step(dtype) * 1.125 * norm
        assert torch.equal(mp.newton_schulz(x[b].cuda()), got[b])


@pytest.mark.parametrize("B,M,N", [(2, 64, 2048), (1, 256, 2048), (3, 120, 130)])
def test_newton_schulz_long_and_narrow_graph(B, M, N):
    """A captured call gives the eager results at every replay, with other work and other inputs in between."""
    g = gen(B + M + N)
    inputs = [grads(g, B, M, N, torch.bfloat16).cuda() for _ in range(3)]
    want = [mp.newton_schulz(x) for x in inputs]
    x = inputs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mp.newton_schulz(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mp.newton_schulz(x)
    for i in (1, 0, 2, 2, 1):
        x.copy_(inputs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(mp.newton_schulz(inputs[i]), want[i])


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("M,N", [(60, 1100), (128, 128), (900, 128), (190, 1300)])
def test_newton_schulz_long_and_narrow_steps(steps, M, N):
    x = grads(gen(steps + M + N), 2, M, N, torch.bfloat16)
    got = mp.newton_schulz(x.cuda(), steps=steps)
    for b in range(2):
        want = mx.newton_schulz(x[b], steps=steps)
        off, norm = torch.linalg.vector_norm(got[b].double().cpu() - want), torch.linalg.vector_norm(want)
        assert off <= mx.half_step(torch.bfloat16) * 1.125 * norm


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("M,N", [(256, 256), (200, 1000), (900, 130), (300, 333)])
@pytest.mark.parametrize("noise", [1e-2, 1e-4])
def test_newton_schulz_near_low_rank(M, N, name, noise):
    """Singular values far below the first ones, which the iteration lifts by a at every step and the roundings of
    the large ones must not drown."""
    dt = mx.TYPES[name]
    x = grads(gen(M + N), 1, M, N, dt, noise=noise, rank=8)[0]
    want = mx.newton_schulz(x)
    got = mp.newton_schulz(x.cuda()).double().cpu()
    off, norm = torch.linalg.vector_norm(got - want), torch.linalg.vector_norm(want)
    assert off <= mx.half_step(dt) * 1.125 * norm


def test_newton_schulz_scales():
    """|G| far below eps, far above 1 and near the ends of bf16; the result keeps its relative accuracy."""
    g = gen(3)
    base = grads(g, 1, 70, 150, torch.float32)[0]
    base = base / torch.linalg.vector_norm(base)
    for scale in (2.0 ** -100, 1e-20, 1e-12, 1e-7, 1e10, 2.0 ** 100):
        x = (base * scale).bfloat16()
        want = mx.newton_schulz(x)
        got = mp.newton_schulz(x.cuda()).double().cpu()
        off, norm = torch.linalg.vector_norm(got - want), torch.linalg.vector_norm(want)
        assert off <= mx.half_step(torch.bfloat16) * 1.125 * norm, scale


@pytest.mark.parametrize("coeffs", [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (4.0, 3.0, 2.0)])
@pytest.mark.parametrize("M,N", [(64, 64), (60, 200)])
def test_newton_schulz_coefficients(coeffs, M, N):
    """Other polynomials: the cubic one, a quintic one, the identity, and two that take the matrix away from the bound
    its number format follows: a power, and one that grows at every step. Those are refused."""
    x = grads(gen(5), 1, M, N, torch.bfloat16)[0]
    if coeffs[0] in (0.0, 4.0):
        with pytest.raises(mp.MpgemmError) as e:
            mp.newton_schulz(x.cuda(), steps=4, coeffs=coeffs)
        assert e.value.status == mp.MPGEMM_ERR_UNSUPPORTED
        return
    want = mx.newton_schulz(x, steps=4, coeffs=coeffs)
    got = mp.newton_schulz(x.cuda(), steps=4, coeffs=coeffs).double().cpu()
    off, norm = torch.linalg.vector_norm(got - want), torch.linalg.vector_norm(want)
    assert off <= mx.half_step(torch.bfloat16) * 1.125 * norm
