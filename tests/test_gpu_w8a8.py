"""The 8-bit integer linear layer on the GPU against 64 bits: quantisation bit for bit, products within the roundings
that the definition has."""
import pytest
import torch

from . import linear_util as lu

pytestmark = pytest.mark.gpu
TYPES = lu.TYPES


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    assert torch.cuda.is_available()
    return mp


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def quantised(mp, x):
    q, s = mp.quantize_i8(x)
    return q.cpu().long(), s.cpu()


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


# ------------------------------------------------------------------ quantisation

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 16), (4, 31), (2, 512), (6, 513), (1, 2048), (3, 2049), (64, 4096), (5, 4100),
                                 (2, 8192), (3, 8200), (2, 20000), (300, 72)])
def test_quantize_bit_for_bit(mp, t, M, K):
    g = gen(M * 7 + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(TYPES[t])
    assert same(quantised(mp, x.cuda()), lu.quantize(x))
    q, s = mp.quantize_i8(x.cuda())
    assert q.stride(0) % 16 == 0 and s.dtype == torch.float32


@pytest.mark.parametrize("t", TYPES)
def test_quantize_ties_and_ends(mp, t):
    dt = TYPES[t]
    # scale 1/8: quotients on every half-way point, and the ends
    x = torch.cat([torch.arange(-127, 128).double() / 8, (torch.arange(-126, 126).double() + 0.5) / 8])
    rows = [x, x * 2.0 ** -6, x * 4, torch.zeros_like(x), -torch.zeros_like(x)]
    tiny = torch.zeros_like(x)
    tiny[3], tiny[4] = lu.smallest(dt) * 100, -lu.smallest(dt) * 3
    rows.append(tiny)
    one = torch.zeros_like(x)
    one[5] = lu.smallest(dt)
    rows.append(one)
    big = torch.zeros_like(x)
    big[7], big[8], big[9] = torch.finfo(dt).max, -torch.finfo(dt).max / 3, 1.0
    rows.append(big)
    x = torch.stack(rows).to(dt)
    got = quantised(mp, x.cuda())
    assert same(got, lu.quantize(x))
    assert not got[0][3].any() and got[1][3] == 0


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_rows_with_no_scale(mp, t, bad):
    x = torch.randn(6, 700, generator=gen(5)).to(TYPES[t])
    x[1, 0], x[4, 699], x[5, 333] = bad, bad, bad
    code, s = quantised(mp, x.cuda())
    want = lu.quantize(x)
    assert torch.equal(torch.isnan(s), torch.tensor([False, True, False, False, True, True]))
    assert torch.equal(code, want[0]) and torch.equal(s[[0, 2, 3]], want[1][[0, 2, 3]])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("layout", ["padded", "anywhere"])
@pytest.mark.parametrize("M,K", [(5, 40), (3, 1000), (2, 4104), (2, 8200)])
def test_quantize_layouts(mp, t, layout, M, K):
    x = torch.randn(M, K, generator=gen(K)).to(TYPES[t])
    assert same(quantised(mp, lu.rows_on_gpu(x, layout)), lu.quantize(x))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (7, 31), (3, 256), (5, 300), (2, 2056), (65, 4100)])
@pytest.mark.parametrize("layout", ["padded", "contiguous", "anywhere"])
def test_dequantize(mp, t, M, K, layout):
    q, s = lu.random_codes(gen(M + K), M, K)
    y = mp.dequantize_i8(*lu.on_gpu((q, s), layout), dtype=TYPES[t])
    assert torch.equal(y.cpu(), (q.float() * s[:, None]).to(TYPES[t]))   # (one fp32 product, one rounding)


# ------------------------------------------------------------------ products

SHAPES = [(1, 1, 1), (1, 17, 16), (1, 64, 300), (2, 33, 256), (3, 100, 4096), (16, 48, 520), (17, 65, 511), (32, 16, 1024), (33, 130, 257),
          (64, 70, 640), (65, 64, 128), (65, 200, 100), (100, 1000, 64), (129, 127, 384), (257, 300, 300), (300, 513, 1100), (520, 260, 16), (700, 900, 2000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("t", TYPES)
def test_held_product(mp, M, N, K, t):
    g = gen(M + 3 * N + 5 * K)
    a, b = lu.random_codes(g, M, K), lu.random_codes(g, N, K)
    bias = torch.randn(N, generator=g).to(TYPES[t]) if (M + N) % 2 else None
    y, mag = lu.scaled(a, b, bias)
    if t == "f16":   # (products up to 128^2 K: scaled to stay finite)
        f = 2.0 ** -13
        a = (a[0], a[1] * f)
        y, mag = lu.scaled(a, b, bias)
    for layout in ("padded", "contiguous", "anywhere"):
        c = mp.gemm_w8a8(*lu.on_gpu(a, layout), *lu.on_gpu(b, layout), bias=None if bias is None else bias.cuda(), dtype=TYPES[t])
        lu.check(c, y, lu.scaled_tol(y, mag, TYPES[t]))


@pytest.mark.parametrize("M,N,K", [(2100, 2050, 130), (1030, 4096, 64), (4096, 300, 192), (2048, 2048, 1040)])
def test_held_product_in_large_tiles(mp, M, N, K):
    """Sizes that take 256 x 256 tiles, ragged ones too; K that ends inside a chunk."""
    for k in (K, K - 3):
        g = gen(M + N + k)
        a, b = lu.random_codes(g, M, k), lu.random_codes(g, N, k)
        y, mag = lu.scaled(a, b)
        c = mp.gemm_w8a8(*lu.on_gpu(a), *lu.on_gpu(b), dtype=torch.bfloat16)
        lu.check(c, y, lu.scaled_tol(y, mag, torch.bfloat16))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 40, 1), (1, 300, 4096), (1, 33, 16384), (1, 64, 17000), (2, 48, 777), (4, 100, 4096), (5, 64, 4096), (16, 32, 1024),
                                   (16, 100, 1030), (30, 70, 600), (64, 64, 100), (65, 100, 100), (200, 300, 515), (300, 520, 2100)])
def test_dynamic_is_quantise_then_held(mp, t, M, N, K):
    g = gen(M * N + K)
    dt = TYPES[t]
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(dt)
    w = lu.quantize(0.02 * torch.randn(N, K, generator=g))
    w = (w[0].to(torch.int8), w[1])
    bias = torch.randn(N, generator=g).to(dt)
    for layout in ("contiguous", "padded", "anywhere"):
        xd, (wq, ws) = lu.rows_on_gpu(x, layout), lu.on_gpu(w, layout)
        y = mp.gemm_w8a8_dyn(xd, wq, ws, bias=bias.cuda())
        assert torch.equal(y, mp.gemm_w8a8(*mp.quantize_i8(xd), wq, ws, bias=bias.cuda(), dtype=dt))
        want, mag = lu.scaled(lu.quantize(x), w, bias)
        lu.check(y, want, lu.scaled_tol(want, mag, dt))


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_a_row_without_scale_is_nan_and_no_other(mp, M):
    g = gen(M)
    x = torch.randn(M, 515, generator=g)
    x[M // 2, 514] = float("nan")
    w = lu.random_codes(g, 70, 515)
    y = mp.gemm_w8a8_dyn(x.bfloat16().cuda(), *lu.on_gpu(w)).cpu()
    assert torch.isnan(y[M // 2]).all()
    assert torch.isfinite(y[[i for i in range(M) if i != M // 2]]).all()


@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (20, 300, 512), (200, 300, 512), (600, 700, 512)])
def test_out_views_are_written_inside_only(mp, M, N, K):
    g = gen(N)
    a, b = lu.on_gpu(lu.random_codes(g, M, K)), lu.on_gpu(lu.random_codes(g, N, K))
    want = mp.gemm_w8a8(*a, *b, dtype=torch.bfloat16)
    for ld, at in ((N + 12, 0), (N + 16, 8), (N + 5, 3)):
        big = torch.full((M + 2, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        view = big[1:M + 1, at:at + N]
        assert mp.gemm_w8a8(*a, *b, out=view).data_ptr() == view.data_ptr()
        assert torch.equal(view, want)
        rest = big.clone()
        rest[1:M + 1, at:at + N] = 7.0
        assert (rest == 7.0).all()


def test_empty(mp):
    q = lambda r, k: (torch.zeros(r, k, dtype=torch.int8, device="cuda"), torch.ones(r, device="cuda"))   # noqa: E731
    bias = torch.randn(6, device="cuda")
    assert mp.gemm_w8a8(*q(0, 8), *q(6, 8)).shape == (0, 6)
    assert mp.gemm_w8a8(*q(5, 8), *q(0, 8)).shape == (5, 0)
    assert torch.equal(mp.gemm_w8a8(*q(5, 0), *q(6, 0), bias=bias), bias.expand(5, 6))
    assert torch.equal(mp.gemm_w8a8_dyn(torch.zeros(70, 0, device="cuda"), *q(6, 0)), torch.zeros(70, 6, device="cuda"))
    codes, s = mp.quantize_i8(torch.zeros(4, 0, device="cuda"))
    assert codes.shape == (4, 0) and torch.equal(s, torch.zeros(4, device="cuda"))
    assert mp.quantize_i8(torch.zeros(0, 9, device="cuda"))[0].shape == (0, 9)


@pytest.mark.parametrize("M", [1, 12, 50, 300])
def test_another_stream_and_a_captured_call(mp, M):
    g = gen(M)
    dt = torch.bfloat16
    xs = [torch.randn(M, 1000, generator=g).to(dt).cuda() for _ in range(3)]
    w = lu.on_gpu(lu.random_codes(g, 200, 1000))
    want = [mp.gemm_w8a8_dyn(x, *w) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mp.gemm_w8a8_dyn(xs[0], *w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mp.gemm_w8a8_dyn(x, *w)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(mp.gemm_w8a8_dyn(xs[i], *w), want[i])


def test_products_of_integers_beyond_fp32(mp):
    """Sums over 2^24 are rounded once, not on the way: one row of equal signs, K = 131071."""
    K = 131071
    a = (torch.full((2, K), -128, dtype=torch.int8), torch.ones(2))
    b = (torch.full((3, K), -128, dtype=torch.int8), torch.ones(3))
    b[0][1, 7] = 127
    for rows in (2, 70):
        aa = (a[0][:1].expand(rows, K).contiguous(), torch.ones(rows))
        y = mp.gemm_w8a8(*lu.on_gpu(aa), *lu.on_gpu(b))
        want, _ = lu.scaled(aa, b)
        assert torch.equal(y.cpu(), want.float())
    with pytest.raises(mp.MpgemmError):
        mp.gemm_w8a8(torch.zeros(1, K + 1, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda"),
                     torch.zeros(1, K + 1, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda"))


# More rows than one launch has threads for, in either direction, and rows behind 2^32 elements.
def test_quantize_of_very_many_rows(mp):
    M, K, at = (1 << 22) + 5, 4104, [0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 1, 1 << 22, (1 << 22) + 4]
    x = torch.zeros(M, K, dtype=torch.float16, device="cuda")
    some = (torch.randn(len(at), K, generator=gen(K)) * 3).half()
    x[at] = some.cuda()
    q, s = mp.quantize_i8(x)
    wq, ws = mp.quantize_i8(some.cuda())
    assert torch.equal(q[at], wq) and torch.equal(s[at], ws)
    assert int((s != 0).sum()) == len(at)
    y = mp.dequantize_i8(q, s, dtype=torch.float16)
    assert torch.equal(y[at], mp.dequantize_i8(wq, ws, dtype=torch.float16))


# So many columns that the workgroups that have quantised the rows go on to further ones.
@pytest.mark.parametrize("M,N,K", [(1, 8193, 700), (1, 20003, 64), (5, 24579, 1000), (8, 16399, 2048)])
@pytest.mark.parametrize("t", lu.TYPES)
def test_quantised_in_the_call_with_many_columns(mp, M, N, K, t):
    dt = lu.TYPES[t]
    g = gen(M + N + K)
    x = torch.randn(M, K, generator=g).to(dt)
    q, s = lu.quantize(torch.randn(N, K, generator=g))
    w = lu.on_gpu((q.to(torch.int8), s))
    bias = torch.randn(N, generator=g).to(dt).cuda()
    y = mp.gemm_w8a8_dyn(x.cuda(), *w, bias=bias)
    want, mag = lu.scaled(lu.quantize(x), (q, s), bias.cpu())
    lu.check(y, want, lu.scaled_tol(want, mag, dt))
    assert torch.equal(y, mp.gemm_w8a8(*mp.quantize_i8(x.cuda()), *w, bias=bias, dtype=dt))


# Large tiles that do not go round the CUs evenly.
@pytest.mark.parametrize("M,N,K", [(2100, 10300, 1030), (4100, 5000, 2048), (777, 23000, 1040)])
def test_product_in_uneven_rounds_of_tiles(mp, M, N, K):
    g = gen(N)
    a, b = (torch.randint(-127, 128, s, generator=g, dtype=torch.int8) for s in ((M, K), (N, K)))
    one = [torch.ones(n, device="cuda") for n in (M, N)]
    c = mp.gemm_w8a8(a.cuda(), one[0], b.cuda(), one[1])
    want = (a.double() @ b.double().t()).float()   # (exact, then one rounding)
    assert torch.equal(c.cpu(), want)
