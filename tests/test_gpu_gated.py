"""The gated feed-forward block on the GPU against 64 bits: forward and backward in 16 bits, the block on 8-bit
integers, and both as they are used together."""
import pytest
import torch

from . import linear_util as lu

pytestmark = pytest.mark.gpu
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ["silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def mp():
    import precision_dense_gemm_tiled_amd as mp
    assert torch.cuda.is_available()
    return mp


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def block(g, M, N, K, dt, size=None):
    """Activations and weights whose products are of order one (a few larger)."""
    size = 1.5 / max(K, 1) ** 0.5 if size is None else size
    x = torch.randn(M, K, generator=g).to(dt)
    return x, (size * torch.randn(N, K, generator=g)).to(dt), (size * torch.randn(N, K, generator=g)).to(dt)


SHAPES = [(1, 1, 1), (1, 40, 8), (1, 17, 300), (1, 64, 4096), (2, 100, 129), (16, 33, 512), (17, 48, 200), (40, 70, 1000), (64, 32, 72), (65, 32, 64),
          (70, 100, 40), (100, 33, 65), (128, 64, 128), (129, 200, 136), (300, 257, 520), (520, 600, 333), (700, 130, 1040)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("t", T16)
def test_forward(mp, M, N, K, t):
    dt = T16[t]
    name = ACTS[(M + N + K) % 3]
    x, wg, wu = block(gen(M + N * 3 + K), M, N, K, dt)
    want, tol = lu.gated(x, wg, wu, name)
    for layout in ("contiguous", "padded", "anywhere"):
        d = [lu.rows_on_gpu(v, layout) for v in (x, wg, wu)]
        h = mp.gemm_gated(*d, act=name)
        h2, g, u = mp.gemm_gated(*d, act=name, keep=True)
        assert torch.equal(h, h2)
        for got, w, e in zip((h, g, u), want, tol):
            lu.check(got, w, lu.rounded_tol(w, e, dt))


@pytest.mark.parametrize("M,N,K", [(2100, 1030, 72), (1024, 2048, 200), (4000, 700, 64)])
def test_forward_in_large_tiles(mp, M, N, K):
    for k in (K, K + 3):
        x, wg, wu = block(gen(M + N + k), M, N, k, torch.bfloat16)
        want, tol = lu.gated(x, wg, wu, "silu")
        for layout in ("contiguous", "padded"):
            got = mp.gemm_gated(*(lu.rows_on_gpu(v, layout) for v in (x, wg, wu)), keep=True)
            for y, w, e in zip(got, want, tol):
                lu.check(y, w, lu.rounded_tol(w, e, torch.bfloat16))


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M", [1, 20, 90])
def test_forward_far_from_zero(mp, name, M):
    """Gates to where the activation has reached its limits, on both sides."""
    dt = torch.bfloat16
    x, wg, wu = block(gen(M), M, 96, 64, dt, size=4.0)
    want, tol = lu.gated(x, wg, wu, name)
    assert want[1].max() > 60 and want[1].min() < -60
    h = mp.gemm_gated(x.cuda(), wg.cuda(), wu.cuda(), act=name)
    lu.check(h, want[0], lu.rounded_tol(want[0], tol[0], dt))


@pytest.mark.parametrize("M", [3, 100])
def test_infinities_and_nan_stay_in_their_rows_and_columns(mp, M):
    x, wg, wu = block(gen(M), M, 80, 200, torch.bfloat16)
    x[1, 5] = float("nan")
    wg[7, 199], wu[9, 0] = float("inf"), float("nan")
    h = mp.gemm_gated(x.cuda(), wg.cuda(), wu.cuda()).cpu()
    assert torch.isnan(h[1]).all() and torch.isnan(h[:, 9]).all()
    clean = h.clone()
    clean[1], clean[:, 7], clean[:, 9] = 0, 0, 0
    assert torch.isfinite(clean).all()


BACK = [(1, 1, 1), (1, 40, 24), (3, 64, 64), (65, 100, 40), (64, 63, 72), (100, 65, 33), (130, 200, 136), (257, 129, 300), (300, 260, 520),
        (777, 100, 130), (70, 700, 260), (520, 64, 1040)]


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("t", T16)
def test_backward(mp, M, N, K, t):
    dt = T16[t]
    name = ACTS[(M + N + K) % 3]
    gg = gen(M * 5 + N + K)
    x, wg, wu = block(gg, M, N, K, dt)
    dh = torch.randn(M, N, generator=gg).to(dt)
    g, u = (x.double() @ wg.double().t()).to(dt), (x.double() @ wu.double().t()).to(dt)
    want = lu.gated_backward(dh, x, wg, wu, g, u, name, dt)
    for layout in ("contiguous", "padded", "anywhere"):
        d = [lu.rows_on_gpu(v, layout) for v in (dh, x, wg, wu, g, u)]
        got = mp.gemm_gated_backward(*d, act=name)
        for y, (w, e) in zip(got, want):
            lu.check(y, w, e)
        dx, none1, none2 = mp.gemm_gated_backward(d[0], None, d[2], d[3], d[4], d[5], act=name, need_dw=False)
        assert none1 is None and none2 is None and torch.equal(dx, got[0])
        none0, dwg, dwu = mp.gemm_gated_backward(d[0], d[1], None, None, d[4], d[5], act=name, need_dx=False)
        assert none0 is None and torch.equal(dwg, got[1]) and torch.equal(dwu, got[2])


@pytest.mark.parametrize("M,N,K", [(2100, 1030, 1100), (520, 2048, 2050), (2048, 1024, 1024)])
def test_backward_in_large_tiles(mp, M, N, K):
    dt = torch.bfloat16
    gg = gen(M)
    x, wg, wu = block(gg, M, N, K, dt)
    dh = torch.randn(M, N, generator=gg).to(dt)
    g, u = (x.double() @ wg.double().t()).to(dt), (x.double() @ wu.double().t()).to(dt)
    got = mp.gemm_gated_backward(*(v.cuda() for v in (dh, x, wg, wu, g, u)))
    for y, (w, e) in zip(got, lu.gated_backward(dh, x, wg, wu, g, u, "silu", dt)):
        lu.check(y, w, e)


@pytest.mark.parametrize("name", ACTS)
def test_backward_where_the_gate_is_far_out(mp, name):
    dt = torch.bfloat16
    M, N, K = 70, 64, 64
    gg = gen(8)
    x, wg, wu = block(gg, M, N, K, dt)
    dh = torch.randn(M, N, generator=gg).to(dt)
    u = torch.randn(M, N, generator=gg).to(dt)
    g = (torch.randn(M, N, generator=gg) * torch.exp(2 * torch.randn(M, N, generator=gg))).to(dt)
    g[0, :4] = torch.tensor([3e38, -3e38, 1e20, -1e20], dtype=dt)
    dh[0, :4] = 0   # (what is multiplied by such a gate's activation)
    got = mp.gemm_gated_backward(*(v.cuda() for v in (dh, x, wg, wu, g, u)), act=name)
    g[0, :4] = 0    # (any finite gate gives the same zeros)
    for y, (w, e) in zip(got, lu.gated_backward(dh, x, wg, wu, g, u, name, dt)):
        lu.check(y, w, e)


@pytest.mark.parametrize("name", ACTS)
def test_gradients_against_differences(mp, name):
    """The derivative of sum(H dH) along random directions of X, Wg and Wu, by central differences in 64 bits."""
    dt = torch.bfloat16
    M, N, K = 80, 96, 72
    gg = gen(3)
    x, wg, wu = block(gg, M, N, K, dt)
    dh = torch.randn(M, N, generator=gg).to(dt)
    _, g, u = mp.gemm_gated(x.cuda(), wg.cuda(), wu.cuda(), act=name, keep=True)
    grads = mp.gemm_gated_backward(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), g, u, act=name)
    at = [v.double() for v in (x, wg, wu)]

    def value(v):
        return ((lu.act(name, v[0] @ v[1].t())[0] * (v[0] @ v[2].t())) * dh.double()).sum()

    for i, grad in enumerate(grads):
        d = torch.randn(at[i].shape, generator=gg, dtype=torch.float64)
        eps = 1e-5
        up, down = [v.clone() for v in at], [v.clone() for v in at]
        up[i] += eps * d
        down[i] -= eps * d
        slope = (value(up) - value(down)) / (2 * eps)
        mine = (grad.double().cpu() * d).sum()
        # G and U rounded (half a step; the slope's change with g is at most 1.2), dG and dU rounded, the gradient rounded: each at most a
        # half step of values whose errors are independent of the direction's signs: 6 of them on the root of the summed squares, six sigma
        scale = (grad.double().cpu() * d).square().sum().sqrt()
        assert (mine - slope).abs() <= 6 * 6 * lu.half_step(dt) * scale


def test_keep_and_out(mp):
    x, wg, wu = (v.cuda() for v in block(gen(1), 90, 70, 64, torch.float16))
    want = mp.gemm_gated(x, wg, wu)
    big = torch.full((92, 80), 5.0, dtype=torch.float16, device="cuda")
    h, g, u = mp.gemm_gated(x, wg, wu, keep=True, out=big[1:91, 3:73])
    assert torch.equal(big[1:91, 3:73], want) and torch.equal(h, want)
    big[1:91, 3:73] = 5.0
    assert (big == 5.0).all()
    # halves of one stacked weight
    w = torch.cat([wg, wu])
    assert torch.equal(mp.gemm_gated(x, w[:70], w[70:]), want)


def test_weights_with_different_strides(mp):
    dt = torch.bfloat16
    gg = gen(2)
    x, wg, wu = block(gg, 100, 64, 48, dt)
    dh, g, u = (torch.randn(100, 64, generator=gg).to(dt) for _ in range(3))
    wide = torch.zeros(64, 80, dtype=dt, device="cuda")
    wide[:, :48] = wu.cuda()
    d = [v.cuda() for v in (dh, x, wg, wu, g, u)]
    want = mp.gemm_gated_backward(*d)
    d[3] = wide[:, :48]
    assert all(torch.equal(a, b) for a, b in zip(mp.gemm_gated_backward(*d), want))
    assert torch.equal(mp.gemm_gated(d[1], d[2], d[3]), mp.gemm_gated(*(v.cuda() for v in (x, wg, wu))))


def test_empty(mp):
    z = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    assert mp.gemm_gated(z(0, 8), z(4, 8), z(4, 8)).shape == (0, 4)
    assert mp.gemm_gated(z(3, 8), z(0, 8), z(0, 8)).shape == (3, 0)
    h, g, u = mp.gemm_gated(z(3, 0), z(4, 0), z(4, 0), keep=True)
    assert not (h.any() or g.any() or u.any()) and h.shape == (3, 4)
    dx, dwg, dwu = mp.gemm_gated_backward(z(0, 4), z(0, 8), z(4, 8), z(4, 8), z(0, 4), z(0, 4))
    assert dx.shape == (0, 8) and dwg.shape == (4, 8) and not dwg.any() and not dwu.any()
    dx, dwg, dwu = mp.gemm_gated_backward(z(3, 0), z(3, 8), z(0, 8), z(0, 8), z(3, 0), z(3, 0))
    assert dx.shape == (3, 8) and not dx.any() and dwg.shape == (0, 8)


# ------------------------------------------------------------------ on integers

@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 40, 300), (1, 64, 4096), (3, 50, 515), (4, 33, 4096), (16, 40, 700), (40, 33, 256), (64, 100, 1000), (65, 32, 128),
                                   (100, 70, 130), (300, 257, 515), (700, 600, 260), (2100, 1030, 200)])
@pytest.mark.parametrize("t", lu.TYPES)
def test_on_integers(mp, M, N, K, t):
    dt = lu.TYPES[t]
    name = ACTS[(M + N + K) % 3]
    g = gen(M + N + K)
    x = torch.randn(M, K, generator=g).to(dt)
    size = 1.5 / K ** 0.5
    w = [lu.quantize(size * torch.randn(N, K, generator=g)) for _ in range(2)]
    w = [(q.to(torch.int8), s) for q, s in w]
    a = lu.quantize(x)
    (pg, mg), (pu, mu) = lu.scaled(a, w[0]), lu.scaled(a, w[1])
    # (three fp32 roundings of each exact sum)
    want, tol = lu.gated_from(pg, pu, 3.01 * 2.0 ** -24 * mg, 3.01 * 2.0 ** -24 * mu, name)
    for layout in ("padded", "contiguous", "anywhere"):
        xd, wg, wu = lu.rows_on_gpu(x, layout), lu.on_gpu(w[0], layout), lu.on_gpu(w[1], layout)
        h = mp.gemm_gated_w8a8_dyn(xd, *wg, *wu, act=name)
        lu.check(h, want[0], lu.rounded_tol(want[0], tol[0], dt))
        assert torch.equal(h, mp.gemm_gated_w8a8(*mp.quantize_i8(xd), *wg, *wu, act=name, dtype=dt))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("M", [130, 300])
def test_a_training_step_then_serving(mp, M):
    """Two steps of a block (gated up-projections, a down-projection by the integer layer's plain form) through an autograd.Function,
    its gradients against 64 bits; then the trained weights are brought into integers and serve one token and a batch."""
    dt = torch.bfloat16
    N, K = 192, 136
    gg = gen(M)
    x, wg, wu = block(gg, M, N, K, dt)
    target = torch.randn(M, N, generator=gg).to(dt)

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, wg, wu):
            h, g, u = mp.gemm_gated(x, wg, wu, keep=True)
            ctx.save_for_backward(x, wg, wu, g, u)
            return h

        @staticmethod
        def backward(ctx, dh):
            return mp.gemm_gated_backward(dh.contiguous(), *ctx.saved_tensors)

    p = [wg.cuda().requires_grad_(), wu.cuda().requires_grad_()]
    xd = x.cuda().requires_grad_()
    for _ in range(2):
        for v in (*p, xd):
            v.grad = None
        h = Gated.apply(xd, *p)
        dh = (h.detach() - target.cuda()) / 8
        h.backward(dh)
        g, u = (v.detach().double().cpu() @ xd.detach().double().cpu().t() for v in p)
        kept = mp.gemm_gated(xd.detach(), p[0].detach(), p[1].detach(), keep=True)[1:]
        want = lu.gated_backward(dh.cpu(), x, p[0].detach().cpu(), p[1].detach().cpu(), kept[0].cpu(), kept[1].cpu(), "silu", dt)
        for grad, (w, e) in zip((xd.grad, p[0].grad, p[1].grad), want):
            lu.check(grad, w, e)
        with torch.no_grad():
            for v in p:
                v -= (0.01 * v.grad).to(dt)
    wd = (torch.randn(K, N, generator=gg) / N ** 0.5).to(dt).cuda()
    held = [mp.quantize_i8(v.detach()) for v in (*p, wd)]
    for rows in (1, M):
        tok = x[:rows].cuda()
        hidden = mp.gemm_gated_w8a8_dyn(tok, *held[0], *held[1])
        y = mp.gemm_w8a8_dyn(hidden, *held[2])
        a, b = lu.quantize(x[:rows]), [(q.cpu(), s.cpu()) for q, s in held]
        (pg, mg), (pu, mu) = lu.scaled(a, b[0]), lu.scaled(a, b[1])
        want, tol = lu.gated_from(pg, pu, 3.01 * 2.0 ** -24 * mg, 3.01 * 2.0 ** -24 * mu, "silu")
        lu.check(hidden, want[0], lu.rounded_tol(want[0], tol[0], dt))
        out, mag = lu.scaled(lu.quantize(hidden.cpu()), b[2])
        lu.check(y, out, lu.scaled_tol(out, mag, dt))


@pytest.mark.parametrize("M", [1, 40, 200])
def test_captured_and_on_another_stream(mp, M):
    dt = torch.bfloat16
    gg = gen(M)
    x0, wg, wu = (v.cuda() for v in block(gg, M, 160, 200, dt))
    xs = [x0, (x0 * 2).contiguous(), (x0 - 1).contiguous()]
    dh = torch.randn(M, 160, generator=gg).to(dt).cuda()

    def step(x, **kw):
        h, g, u = mp.gemm_gated(x, wg, wu, keep=True, **kw)
        return [h, g, u, *mp.gemm_gated_backward(dh, x, wg, wu, g, u, **kw)]

    want = [step(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(xs[1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(x)
    for i in (1, 2, 0, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(step(xs[i]), want[i]))


# Long sums into few columns, and tiles whose second half has no rows, captured where nothing is mapped behind the
# operands: stages past the last one and halves without rows read nothing.
@pytest.mark.parametrize("M,N,K", [(3712, 8576, 384), (1856, 832, 640), (896, 256, 1152), (65, 7680, 64), (70, 333, 129)])
def test_backward_of_long_sums_captured(mp, M, N, K):
    dt = torch.bfloat16
    gg = torch.Generator(device="cuda").manual_seed(N)
    torch.cuda.empty_cache()
    dh, x, wg, wu, g, u = (torch.randn(*s, generator=gg, device="cuda").to(dt) for s in ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N)))
    want = mp.gemm_gated_backward(dh, x, wg, wu, g, u)
    if M < 1000:
        for y, (w, e) in zip(want, lu.gated_backward(*(v.cpu() for v in (dh, x, wg, wu, g, u)), "silu", dt)):
            lu.check(y, w, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = mp.gemm_gated_backward(dh, x, wg, wu, g, u)
    torch.cuda.empty_cache()
    for _ in range(3):
        for y in held:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert all(torch.equal(a, b) for a, b in zip(mp.gemm_gated_backward(dh, x, wg, wu, g, u), want))


# Rows of more than 2^23 bytes, which the products across k take from a copy, and steps of 2^25 bytes.
@pytest.mark.parametrize("K", [5_000_001, (1 << 24) - 3])
def test_backward_with_very_long_rows(mp, K):
    M, N, dt = 66, 3, torch.bfloat16
    gg = torch.Generator(device="cuda").manual_seed(K)
    dh, x, wg, wu, g, u = (torch.randn(*s, generator=gg, device="cuda", dtype=dt) for s in ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N)))
    got = mp.gemm_gated_backward(dh, x, wg, wu, g, u)
    for k in (slice(0, 300), slice(K // 2, K // 2 + 200), slice(K - 300, K)):
        want = lu.gated_backward(*(v.cpu() for v in (dh, x[:, k], wg[:, k], wu[:, k], g, u)), "silu", dt)
        for y, (w, e) in zip(got, want):
            lu.check(y[:, k], w, e)


# So many columns that the workgroups that have quantised the rows go on to further ones.
@pytest.mark.parametrize("M,N,K", [(1, 12291, 260), (3, 4100, 515), (4, 9001, 4096), (7, 16399, 130)])
@pytest.mark.parametrize("t", lu.TYPES)
def test_on_integers_with_many_columns(mp, M, N, K, t):
    test_on_integers(mp, M, N, K, t)


# Rows 2^23 bytes apart and more: above 32 rows from a copy, below as they are.
@pytest.mark.parametrize("M", [2, 20, 70])
def test_rows_far_apart(mp, M):
    K, ld = 72, 4_200_000
    gg = torch.Generator(device="cuda").manual_seed(M)
    far = lambda rows: torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")[:, :K].copy_(torch.randn(rows, K, generator=gg, device="cuda"))  # noqa: E731
    x, wg, wu = far(M), far(40), far(40)
    near = [v.contiguous() for v in (x, wg, wu)]
    h, g, u = mp.gemm_gated(x, wg, wu, keep=True)
    assert all(torch.equal(a, b) for a, b in zip((h, g, u), mp.gemm_gated(*near, keep=True)))
    dh = torch.randn(M, 40, generator=gg, device="cuda").bfloat16()
    got = mp.gemm_gated_backward(dh, x, wg, wu, g, u)
    assert all(torch.equal(a, b) for a, b in zip(got, mp.gemm_gated_backward(dh, *near, g, u)))
    q, s = mp.quantize_i8(x)
    qn, sn = mp.quantize_i8(near[0])
    assert torch.equal(q, qn) and torch.equal(s, sn)


# Calls that share the handle, side by side on two streams, each with its own scratch memory.
def test_two_streams_at_once(mp):
    dt = torch.bfloat16
    gg = gen(5)
    x, wg, wu = (v.cuda() for v in block(gg, 300, 200, 136, dt))
    dh = torch.randn(300, 200, generator=gg).to(dt).cuda()
    t = torch.randn(3, 521, generator=gg).to(dt).cuda()
    w = [mp.quantize_i8(torch.randn(5000, 521, generator=gg).cuda()) for _ in range(2)]

    def train(**kw):
        h, g, u = mp.gemm_gated(x, wg, wu, keep=True, **kw)
        return [h, *mp.gemm_gated_backward(dh, x, wg, wu, g, u, **kw)]

    def serve(**kw):
        return [mp.gemm_gated_w8a8_dyn(t, *w[0], *w[1], **kw), mp.gemm_w8a8_dyn(x, *mp.quantize_i8(wg, **kw), **kw)]

    want = [train(), serve()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i in range(8):
        for k, f in enumerate((train, serve)):
            got[(i + k) % 2].append((k, f(stream=streams[(i + k) % 2])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for side in got for k, v in side for a, b in zip(v, want[k]))


# Large tiles that do not go round the CUs evenly.
@pytest.mark.parametrize("M,N,K", [(2100, 5200, 600), (1800, 4500, 1030), (4097, 2200, 520)])
def test_forward_in_uneven_rounds_of_tiles(mp, M, N, K):
    dt = torch.bfloat16
    x, wg, wu = block(gen(N), M, N, K, dt)
    got = mp.gemm_gated(x.cuda(), wg.cuda(), wu.cuda(), keep=True)
    for y, w, e in zip(got, *lu.gated(x, wg, wu, "silu")):
        lu.check(y, w, lu.rounded_tol(w, e, dt))


# The C call with any of the three gradients left out.
@pytest.mark.parametrize("M,N,K", [(70, 100, 136), (300, 520, 264)])
def test_backward_of_some_gradients(mp, M, N, K):
    dt = torch.bfloat16
    gg = torch.Generator(device="cuda").manual_seed(M)
    dh, x, wg, wu, g, u = (torch.randn(*s, generator=gg, device="cuda").to(dt) for s in ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N)))
    want = mp.gemm_gated_backward(dh, x, wg, wu, g, u)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(mp.mpgemm_run_gated_backward_workspace(M, N, K, 1, cus), dtype=torch.uint8, device="cuda")
    for take in range(1, 8):
        out = [torch.empty_like(v) if take >> i & 1 else None for i, v in enumerate(want)]
        p = [None if v is None else v.data_ptr() for v in out]
        assert mp.mpgemm_run_gated_backward(mp.default_handle(0), M, N, K, 1, 0, dh.data_ptr(), N, x.data_ptr(), K, wg.data_ptr(), K, wu.data_ptr(), K,
                                            g.data_ptr(), N, u.data_ptr(), N, p[0], K, p[1], K, p[2], K, ws.data_ptr(), ws.numel(),
                                            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert all(v is None or torch.equal(v, w) for v, w in zip(out, want))
