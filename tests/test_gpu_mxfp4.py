"""MXFP4 on the GPU against the 64-bit definitions of tests/mx_util.py:
codes and scales bit for bit, products within the stated roundings."""
import pytest
import torch

import precision_dense_gemm_tiled_amd as mp

from . import mx_util as mx

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def some(g, M, K, dtype):
    """Normal values over many binades, with zeros, a row and a block of zeros."""
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-12, 9, (M, K), generator=g).float())
    x = torch.where(torch.rand(M, K, generator=g) < 0.1, torch.zeros(()), x)
    if M > 2:
        x[M // 2] = 0
    x[0, 32:64] = 0
    return x.to(dtype)


# ---------------------------------------------------------------- quantisation

SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 4096), (2, 64), (3, 257), (31, 8), (32, 128), (33, 130), (64, 520),
          (127, 129), (128, 128), (129, 127), (160, 72), (333, 1000), (1000, 96)]


@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_both(M, K, name):
    x = some(gen(M * 7919 + K), M, K, mx.TYPES[name])
    q, s, qt, st = mp.quantize_mxfp4_both(x.cuda())
    for (a, b), (wa, wb) in (((q, s), mx.quantize(x)), ((qt, st), mx.quantize(x.t()))):
        assert torch.equal(b.cpu(), wb)
        assert torch.equal(a.cpu(), wa)
    q2, s2 = mp.quantize_mxfp4(x.cuda())
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_quantize_every_value(name):
    """Every 16-bit pattern, in blocks led by values of several sizes (every rounding border and tie of the type),
    NaN and infinities among them."""
    allv = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(mx.TYPES[name])
    rows = [allv.reshape(-1, 32)]
    lead = torch.tensor([2.0 ** e for e in range(-14, 15)]).to(mx.TYPES[name])
    fin = allv[torch.isfinite(allv)]
    for v in lead:
        x = torch.where(fin.abs() <= v * 1.75, fin, torch.zeros_like(fin))
        x = torch.cat([x, x.new_zeros((-len(x)) % 31)]).reshape(-1, 31)
        rows.append(torch.cat([torch.full((len(x), 1), float(v)).to(x.dtype), x], dim=1))
    x = torch.cat(rows)
    q, s, qt, st = mp.quantize_mxfp4_both(x.cuda())
    wq, ws = mx.quantize(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)
    wq, ws = mx.quantize(x.t())
    assert torch.equal(st.cpu(), ws) and torch.equal(qt.cpu(), wq)


def test_quantize_extremes():
    tiny, big = 2.0 ** -149, torch.finfo(torch.float32).max
    x = torch.zeros(8, 32)
    x[0, 3], x[1, 4], x[2, 5], x[2, 6] = tiny, big, big, -big
    x[3] = -0.0
    x[4, 0], x[5, 31], x[6, 7] = float("nan"), float("inf"), -float("inf")
    x[7, :8] = torch.tensor([2.0 ** -126, 2.0 ** -127, 2.0 ** -128, 1.5 * 2.0 ** -129, 2.0 ** -129, 2.0 ** -130, -2.0 ** -128, 0])
    q, s = mp.quantize_mxfp4(x.cuda())
    wq, ws = mx.quantize(x)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)
    y = mp.dequantize_mxfp4(q, s, 32).cpu()
    assert torch.isnan(y[4:7]).all() and torch.isfinite(y[[0, 1, 2, 3, 7]]).all()
    assert torch.equal(y[[0, 1, 2, 3, 7]].double(), mx.values(wq, ws, 32)[[0, 1, 2, 3, 7]])


@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("offset,ld", [(0, 96), (1, 97), (8, 104), (3, 101)])
def test_quantize_views(offset, ld, name):
    M, K = 70, 90
    base = some(gen(offset), 1, M * ld + 16, mx.TYPES[name])[0]
    x = torch.as_strided(base.cuda(), (M, K), (ld, 1), offset)
    q, s, qt, st = mp.quantize_mxfp4_both(x)
    for (a, b), (wa, wb) in (((q, s), mx.quantize(x.cpu())), ((qt, st), mx.quantize(x.cpu().t()))):
        assert torch.equal(b.cpu(), wb) and torch.equal(a.cpu(), wa)


def test_quantize_writes_nothing_past_its_blocks():
    """Raw call into wider buffers: the bytes past the blocks keep their values."""
    M, K = 70, 130
    x = some(gen(5), M, K, torch.bfloat16).cuda()
    nbk, nbm = 5, 3
    q = torch.full((M, 16 * nbk + 32), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((M, 16), 9, dtype=torch.uint8, device="cuda")
    qt = torch.full((K, 16 * nbm + 16), 7, dtype=torch.uint8, device="cuda")
    st = torch.full((K, 32), 9, dtype=torch.uint8, device="cuda")
    rc = mp.mpgemm_quantize_mxfp4(mp.default_handle(), M, K, mp.MPGEMM_TYPE_BF16, x.data_ptr(), K, q.data_ptr(),
                                  q.stride(0), s.data_ptr(), 16, qt.data_ptr(), qt.stride(0), st.data_ptr(), 32,
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    wq, ws = mx.quantize(x.cpu())
    wqt, wst = mx.quantize(x.cpu().t())
    assert torch.equal(q[:, :16 * nbk].cpu(), wq) and torch.equal(s[:, :nbk].cpu(), ws)
    assert torch.equal(qt[:, :16 * nbm].cpu(), wqt) and torch.equal(st[:, :nbm].cpu(), wst)
    assert (q[:, 16 * nbk:] == 7).all() and (s[:, nbk:] == 9).all()
    assert (qt[:, 16 * nbm:] == 7).all() and (st[:, nbm:] == 9).all()


@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
def test_dequantize_every_code_and_scale(name):
    q = torch.arange(256, dtype=torch.uint8).reshape(1, 256).repeat(256, 1)   # 512 codes = 16 blocks
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    K = 509
    y = mp.dequantize_mxfp4(*mx.on_gpu((q, s)), K, mx.TYPES[name]).cpu()
    want = mx.values(q, s, K)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(y[fine], want[fine].float().to(mx.TYPES[name]))
    assert torch.equal(torch.signbit(y[fine]), torch.signbit(want[fine]))


# ---------------------------------------------------------------- products

def product(A, B, K):
    a, b = mx.values(*A, K), mx.values(*B, K)
    return a @ b.t(), a.abs() @ b.abs().t()


GEMMS = [(1, 1, 1), (1, 16, 32), (1, 17, 4096), (2, 5, 33), (15, 40, 600), (16, 64, 8192), (17, 31, 512), (32, 48, 2080),
         (33, 100, 1000), (64, 64, 64), (64, 130, 4000), (65, 64, 32), (65, 3, 257), (100, 100, 100), (128, 128, 256),
         (130, 257, 288), (300, 70, 2100), (70, 64, 8192), (66, 65, 6000), (512, 512, 512), (1000, 520, 777)]


@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm(M, N, K, name):
    g = gen(M + 31 * N + 17 * K)
    A, B = mx.random_held(g, M, K), mx.random_held(g, N, K)
    dt = mx.TYPES[name]
    bias = torch.randn(N, generator=g).to(dt)
    y, t = product(A, B, K)
    big = torch.finfo(dt).max
    A2, B2 = mx.on_gpu(A), mx.on_gpu(B)
    y = torch.where(y.abs() > big, torch.full_like(y, float("inf")) * y.sign(), y)
    fin = torch.isfinite(y)
    got = mp.gemm_mxfp4(*A2, *B2, K, dtype=dt)
    assert got.dtype == dt
    mx.check(torch.where(fin.cuda(), got, torch.zeros((), dtype=dt, device="cuda")),
             torch.where(fin, y, torch.zeros(())).double(), mx.gemm_tol(torch.where(fin, y, torch.zeros(())), t, (K + 31) // 32, dt))
    again = mp.gemm_mxfp4(*A2, *B2, K, dtype=dt)
    assert torch.equal(got, again)
    yb = y + bias.double()
    got = mp.gemm_mxfp4(*A2, *B2, K, bias=bias.cuda(), dtype=dt)
    mx.check(torch.where(fin.cuda(), got, torch.zeros((), dtype=dt, device="cuda")),
             torch.where(fin, yb, torch.zeros(())).double(),
             mx.gemm_tol(torch.where(fin, yb, torch.zeros(())), t + bias.double().abs(), (K + 31) // 32, dt))


# one tile of each shape, whole and ragged, and the last workgroup past both edges
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 288), (2048, 4096, 256), (4097, 4000, 1056), (2049, 2100, 520),
                                   (4000, 2050, 96), (1500, 2600, 2100)])
def test_gemm_large_tiles(M, N, K):
    """Sizes that fill the chip with the larger tiles; checked against a 64-bit product of random columns (every
    output enters)."""
    g = gen(M + N + K)
    A, B = mx.random_held(g, M, K), mx.random_held(g, N, K)
    got = mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), K).double().cpu()
    y, t = product(A, B, K)
    mx.check(got, y, mx.gemm_tol(y, t, (K + 31) // 32, torch.float32))


def test_gemm_exact_sums():
    """Small whole numbers: every partial sum is exact in fp32, so the result is too, in every kernel."""
    g = gen(3)
    for M, N, K in [(5, 33, 500), (40, 64, 1000), (200, 300, 700), (1100, 4096, 512), (4096, 4096, 544)]:
        A, B = mx.random_held(g, M, K, spread=1), mx.random_held(g, N, K, spread=1)
        y, _ = product(A, B, K)
        assert torch.equal(mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), K).double().cpu(), y)


@pytest.mark.parametrize("M", [3, 40, 200])
def test_nan_scales_and_sizes(M):
    """A NaN block makes its row (or column) NaN and nothing else; scale bytes past a row's end (255 here) do
    nothing."""
    g = gen(M)
    N, K = 96, 900
    A, B = mx.random_held(g, M, K), mx.random_held(g, N, K)
    A[1][1, 28] = 255
    B[1][5, 3] = 255
    y, t = product(A, B, K)
    assert int(torch.isnan(y).sum()) == M + N - 1
    mx.check(mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), K), y, mx.gemm_tol(y, t, 29, torch.float32))


def test_extreme_scales():
    """Products whose scales cancel: 2^-127 against 2^127, and results in the top binades."""
    A = (torch.full((4, 16), 0x22, dtype=torch.uint8), torch.tensor([[0], [254], [10], [200]], dtype=torch.uint8))
    B = (torch.full((4, 16), 0x22, dtype=torch.uint8), torch.tensor([[254], [0], [244], [54]], dtype=torch.uint8))
    got = mp.gemm_mxfp4(*mx.on_gpu(A), *mx.on_gpu(B), 32).cpu().double()
    want = 32 * torch.exp2(A[1].double() + B[1].double().t() - 254)
    for i, j in [(0, 0), (1, 1), (2, 2), (3, 3), (0, 2), (3, 1)]:
        assert got[i, j] == want[i, j]
    assert torch.isinf(got[1, 0])   # 2^127 * 2^127


@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 32), (1, 1000, 2100), (7, 100, 33), (16, 130, 1000), (17, 40, 2100), (33, 5000, 96),
                                   (64, 72, 4096), (65, 66, 67), (333, 500, 2100), (700, 1030, 520)])
def test_dyn(M, N, K, name):
    g = gen(M + N + K)
    dt = mx.TYPES[name]
    x = some(g, M, K, dt)
    W = mx.random_held(g, N, K, spread=1)
    bias = torch.randn(N, generator=g).to(dt)
    A = mx.quantize(x)
    y, t = product(A, W, K)
    y, t = y + bias.double(), t + bias.double().abs()
    got = mp.gemm_mxfp4_dyn(x.cuda(), *mx.on_gpu(W), bias=bias.cuda())
    fin = y.abs() < torch.finfo(dt).max / 2
    z = torch.zeros(())
    mx.check(torch.where(fin, got.cpu().double(), z.double()), torch.where(fin, y, z.double()),
             mx.gemm_tol(torch.where(fin, y, z.double()), t, (K + 31) // 32, dt))
    # the same bits as quantising first
    q, s = mp.quantize_mxfp4(x.cuda())
    assert torch.equal(got, mp.gemm_mxfp4(q, s, *mx.on_gpu(W), K, bias=bias.cuda(), dtype=dt))


def test_dyn_nan_and_views():
    g = gen(11)
    for M in (4, 90):
        base = some(g, M, 203, torch.float16)
        base[2, 40] = float("inf")
        base[3, 170] = float("nan")
        x = base.cuda()[:, 3:203]
        W = mx.random_held(g, 50, 200, spread=1)
        out = torch.full((M, 64), 7.0, dtype=torch.float16, device="cuda")
        got = mp.gemm_mxfp4_dyn(x, *mx.on_gpu(W), out=out[:, 5:55])
        y, t = product(mx.quantize(x.cpu()), W, 200)
        assert torch.isnan(y[2:4]).all()
        mx.check(got, y, mx.gemm_tol(torch.nan_to_num(y), torch.nan_to_num(t), 7, torch.float16))
        assert (out[:, :5] == 7).all() and (out[:, 55:] == 7).all()


def test_empty():
    z = torch.zeros
    dev = dict(device="cuda", dtype=torch.float16)
    W = mx.on_gpu(mx.random_held(gen(1), 40, 64))
    assert mp.gemm_mxfp4_dyn(z((0, 64), **dev), *W).shape == (0, 40)
    W0 = (z((0, 32), device="cuda", dtype=torch.uint8), z((0, 2), device="cuda", dtype=torch.uint8))
    assert mp.gemm_mxfp4_dyn(z((3, 64), **dev), *W0).shape == (3, 0)
    K0 = (z((40, 0), device="cuda", dtype=torch.uint8), z((40, 0), device="cuda", dtype=torch.uint8))
    bias = torch.arange(40, **dev)
    assert torch.equal(mp.gemm_mxfp4_dyn(z((3, 0), **dev), *K0, bias=bias), bias.expand(3, 40))
    assert not mp.gemm_mxfp4_dyn(z((100, 0), **dev), *K0).any()
    q, s = mp.quantize_mxfp4(z((0, 64), **dev))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    q, s = mp.quantize_mxfp4(z((3, 0), **dev))
    assert q.shape == (3, 0) and mp.dequantize_mxfp4(q, s, 0).shape == (3, 0)
    # no tokens: a weight gradient of zeros; no outputs: an input gradient of zeros
    held = lambda r, k: mx.on_gpu(mx.random_held(gen(2), r, k))   # noqa: E731
    dx, dw = mp.gemm_mxfp4_backward(z((0, 64), **dev), *held(48, 64), *(z((48, 0), device="cuda", dtype=torch.uint8),) * 2)
    assert dx.shape == (0, 48) and dw.shape == (64, 48) and not dw.any()
    dx, dw = mp.gemm_mxfp4_backward(z((5, 0), **dev), *(z((48, 0), device="cuda", dtype=torch.uint8),) * 2, *held(48, 5))
    assert dx.shape == (5, 48) and not dx.any() and dw.shape == (0, 48)


# ---------------------------------------------------------------- backward

@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 96), (33, 100, 70), (64, 32, 300), (257, 130, 520), (777, 200, 136),
                                   (4000, 64, 64)])
def test_backward(M, N, K, name):
    g = gen(M + N + K)
    dt = mx.TYPES[name]
    dy = (torch.randn(M, N, generator=g) * torch.exp2(torch.randint(-6, 3, (M, 1), generator=g).float())).to(dt)
    WT, XT = mx.random_held(g, K, N, spread=1), mx.random_held(g, K, M, spread=1)
    dx, dw = mp.gemm_mxfp4_backward(dy.cuda(), *mx.on_gpu(WT), *mx.on_gpu(XT))
    assert dx.dtype == dt and dw.dtype == torch.float32
    y, t = product(mx.quantize(dy), WT, N)
    mx.check(dx, y, mx.gemm_tol(y, t, (N + 31) // 32, dt))
    y, t = product(mx.quantize(dy.t()), XT, M)
    mx.check(dw, y, mx.gemm_tol(y, t, (M + 31) // 32, torch.float32))
    only_x, none = mp.gemm_mxfp4_backward(dy.cuda(), *mx.on_gpu(WT), None, None, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = mp.gemm_mxfp4_backward(dy.cuda(), None, None, *mx.on_gpu(XT), need_dx=False)
    assert none is None and torch.equal(only_w, dw)


def test_backward_against_differences():
    """Values that MXFP4 holds exactly, so that the layer is linear in each operand and a difference quotient of the
    library's own forward pass is its gradient: L = sum(dY * gemm(X, W))."""
    g = gen(8)
    M, N, K = 64, 96, 64
    pick = lambda r, c: mx.GRID[torch.randint(0, 7, (r, c), generator=g)] * torch.where(torch.rand(r, c, generator=g) < 0.5, -1, 1)  # noqa: E731
    x, w, dy = pick(M, K), pick(N, K), pick(M, N)
    for m in (x, w, dy):   # every block of 32, along rows and columns, holds a 4: scale 1
        m[::32, :] = 4.0
        m[:, ::32] = 4.0
    half = torch.float16
    wt = mp.quantize_mxfp4_both(w.to(half).cuda())[2:]
    xt = mp.quantize_mxfp4_both(x.to(half).cuda())[2:]
    dx, dw = mp.gemm_mxfp4_backward(dy.to(half).cuda(), *wt, *xt)

    def loss(x, w):
        a, b = mp.quantize_mxfp4(x.float().cuda()), mp.quantize_mxfp4(w.float().cuda())
        return (mp.gemm_mxfp4(*a, *b, K).double().cpu() * dy).sum().item()

    base = loss(x, w)
    for i, j in [(0, 1), (5, 33), (40, 63), (63, 17)]:
        for m, grad in ((x, dx), (w, dw)):
            e = m.clone()
            step = 1.0 if abs(e[i, j]) < 3 else -1.0   # stays on the grid
            e[i, j] = (3.0 if e[i, j] == 4 else 2.0 if e[i, j] == 3 else -2.0 if e[i, j] == -3 else e[i, j] + step * 0.5
                       if abs(e[i, j]) < 2 else 1.5)
            h = (e[i, j] - m[i, j]).item()
            quotient = ((loss(e, w) if m is x else loss(x, e)) - base) / h
            assert abs(quotient - grad[i, j].item()) <= mx.half_step(half) * abs(quotient) + 1e-9


# ---------------------------------------------------------------- streams, graphs

def test_other_stream_and_shared_handle():
    g = gen(4)
    W = mx.on_gpu(mx.random_held(g, 300, 2048))
    xs = [torch.randn(m, 2048, generator=g).half().cuda() for m in (8, 100, 300)]
    want = [mp.gemm_mxfp4_dyn(x, *W) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [None] * 3
    for _ in range(20):
        for i, (x, s) in enumerate(zip(xs, streams)):
            got[i] = mp.gemm_mxfp4_dyn(x, *W, stream=s) if i else mp.gemm_mxfp4_dyn(x, *W, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 48, 200])
def test_graph(M):
    """Forward and backward in one captured graph, replayed on new inputs between eager calls."""
    g = gen(M)
    N, K = 264, 1056
    w = (0.05 * torch.randn(N, K, generator=g)).half().cuda()
    x = torch.randn(M, K, generator=g).half().cuda()
    dy = torch.randn(M, N, generator=g).half().cuda()
    bias = torch.randn(N, generator=g).half().cuda()

    def step():
        wq, ws, wtq, wts = mp.quantize_mxfp4_both(w)
        y = mp.gemm_mxfp4_dyn(x, wq, ws, bias=bias)
        xt = mp.quantize_mxfp4_both(x)[2:]
        return (y,) + mp.gemm_mxfp4_backward(dy, wtq, wts, *xt)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        x.copy_(torch.randn(M, K, generator=g).half())
        dy.copy_(torch.randn(M, N, generator=g).half())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
