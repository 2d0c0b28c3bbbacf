"""Calls of the 8-bit integer layer and the gated block at the ends of what they take: single rows of great length, held
matrices that are saved and loaded, gates far below zero, gradients that only one weight needs."""
import math

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


EPS = 2.0 ** -23


def act64(name, v):
    """The activation and its derivative in 64 bits, to their last digits far below zero (there 1 + tanh z is taken as 2 sigmoid(2 z))."""
    if name != "gelu_tanh":
        return lu.act(name, v)
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (v + 0.044715 * v ** 3))
    return v * s, s + v * s * (1 - s) * c * (1 + 3 * 0.044715 * v * v)


def act_rel(name, v):
    """What the fp32 evaluation of an activation may be off by, relative to its value. silu: the exponent's argument |v| with a rounded constant
    and product (1 EPS together), exp2 and the reciprocal 1 EPS each, the sum and the product half a one each. gelu_tanh: its argument z has nine
    roundings of half an EPS. gelu: the normal distribution at v as an exponential whose argument v^2 / 2 has three roundings of
    half an EPS, exp2 and a reciprocal (1 EPS each, 1 for the reciprocal's argument), a polynomial (its fit, its coefficients' and its steps'
    roundings: 3.5) and three products."""
    a = v.abs()
    if name == "silu":
        return (a + 4) * EPS
    if name == "gelu_tanh":
        return (4.5 * 1.59577 * (a + 0.044715 * a ** 3) + 4) * EPS
    return (8 + 0.75 * v * v) * EPS


# Far below zero an activation is small beside its gate and keeps its digits all the same. Integers with one code for each gate:
# G = -1 |v| 1, U = -1 |v| (1 / 2), H = act(v) v / 2.
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 4, 20, 32, 600])
def test_activations_far_below_zero(mp, name, M):
    v = -torch.cat([torch.linspace(0.01, 9, max(M - 1, 1)), torch.tensor([5.5])])[-M:]
    N = 40
    a = torch.full((M, 1), -1, dtype=torch.int8, device="cuda"), -v.cuda()
    one = torch.ones(N, 1, dtype=torch.int8, device="cuda")
    h = mp.gemm_gated_w8a8(*a, one, torch.ones(N, device="cuda"), one, torch.full((N,), 0.5, device="cuda"), act=name, dtype=torch.float32)
    v = v.double()[:, None].expand(M, N)
    want = act64(name, v)[0] * v / 2
    lu.check(h, want, want.abs() * (act_rel(name, v) + 0.51 * EPS) + 2.0 ** -126)


# The same in 16 bits, with the backward pass: tokens are rows of the identity, so that dWg and dWu are dG and dU as they were rounded.
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gradients_far_below_zero(mp, name):
    dt, M, N = torch.bfloat16, 64, 48
    g = -torch.linspace(0.01, 9, M * N).reshape(M, N).to(dt)
    one = torch.ones(M, N, dtype=dt)
    dh, x, gd = one.cuda(), torch.eye(M, dtype=dt, device="cuda"), g.cuda()
    dx, dwg, dwu = mp.gemm_gated_backward(dh, x, None, None, gd, dh, act=name, need_dx=False)
    v = g.double()
    a, slope = act64(name, v)
    lu.check(dwu.t(), a, lu.rounded_tol(a, a.abs() * act_rel(name, v), dt))
    # the slope is a sum: the sigmoid (a over v) and what is left, by the same roundings and four more products and sums
    part = (a / v).abs()
    err = (part + (slope - a / v).abs()) * (act_rel(name, v) + 4 * EPS)
    if name == "silu":
        err = err + part * 2 * EPS * v.abs()      # (1 - s, off by 1 EPS, times v)
    if name == "gelu_tanh":
        err = err + part * 2 * EPS * (v.abs() * 1.6 * (1 + 0.134145 * v * v))
    lu.check(dwg.t(), slope, lu.rounded_tol(slope, err, dt))
    # forward: G = g exactly, U = 1
    wg, wu = torch.zeros(N, 8, dtype=dt), torch.zeros(N, 8, dtype=dt)
    wg[:, 0] = g[0]
    wu[:, 1] = 1
    for rows in (1, 3, 20, 100):
        t = torch.zeros(rows, 8, dtype=dt)
        t[:, :2] = 1
        h = mp.gemm_gated(t.cuda(), wg.cuda(), wu.cuda(), act=name)
        want = a[:1].expand(rows, N)
        lu.check(h, want, lu.rounded_tol(want, want.abs() * act_rel(name, v[:1]), dt))


# Gates that are not finite: the derivative of NaN is NaN, at the ends it is 0 and 1.
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slopes_of_gates_that_are_not_finite(mp, name):
    dt = torch.bfloat16
    g = torch.tensor([[float("nan"), float("inf"), -float("inf"), 3e38, -3e38, 0.0, -0.0, 1.0]], dtype=dt, device="cuda")
    one = torch.ones_like(g)
    dx, dwg, dwu = mp.gemm_gated_backward(one, torch.ones(1, 8, dtype=dt, device="cuda"), None, None, g, one, act=name, need_dx=False)
    want = lu.act(name, torch.tensor([1.0]))[1].to(dt).item()
    got = dwg[:, 0].tolist()
    assert math.isnan(got[0]) and got[1:7] == [1.0, 0.0, 1.0, 0.0, 0.5, 0.5] and abs(got[7] - want) <= 2.0 ** -8 * want
    act = dwu[:, 0].tolist()
    assert math.isnan(act[0]) and act[1] == float("inf") and act[3] > 2.9e38 and act[4:7] == [0.0, 0.0, 0.0]


# Forward mode: a tangent would be lost in the call itself; inside an autograd.Function the call runs and the function's jvp gives it.
def test_tangents_through_an_autograd_function(mp):
    dt = torch.bfloat16
    gg = torch.Generator().manual_seed(1)
    x, wg, wu, v = (torch.randn(6, 16, generator=gg).to(dt).cuda() for _ in range(4))

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(x):
            return mp.gemm_gated(x, wg, wu)

        @staticmethod
        def setup_context(ctx, inputs, output):
            ctx.save_for_forward(inputs[0])

        @staticmethod
        def jvp(ctx, t):
            x, = ctx.saved_tensors
            return (mp.gemm_gated(x + t, wg, wu) - mp.gemm_gated(x - t, wg, wu)) / 2

    fw = torch.autograd.forward_ad
    with fw.dual_level():
        d = fw.make_dual(x, v)
        with pytest.raises(RuntimeError, match="tangent"):
            mp.gemm_gated(d, wg, wu)
        y, t = fw.unpack_dual(Gated.apply(d))
    assert torch.equal(y, mp.gemm_gated(x, wg, wu))
    assert torch.equal(t, (mp.gemm_gated(x + v, wg, wu) - mp.gemm_gated(x - v, wg, wu)) / 2)


def backward_call(mp, t, want, ws, act=0):
    """The C call on dH, X, Wg, Wu, G and U (contiguous, bf16) for those of dX, dWg and dWu that are wanted; its launches follow the
    current stream."""
    dh, x, wg, wu, g, u = t
    (M, N), K = dh.shape, x.shape[1]
    out = [torch.full(s, 7.0, dtype=dh.dtype, device="cuda") if y else None for y, s in zip(want, ((M, K), (N, K), (N, K)))]
    p = [None if v is None else v.data_ptr() for v in out]

    def run():
        assert mp.mpgemm_run_gated_backward(mp.default_handle(0), M, N, K, 1, act, dh.data_ptr(), N, x.data_ptr(), K, wg.data_ptr(), K, wu.data_ptr(), K,
                                            g.data_ptr(), N, u.data_ptr(), N, p[0], K, p[1], K, p[2], K, ws.data_ptr(), ws.numel(),
                                            torch.cuda.current_stream().cuda_stream) == 0
    return run, out


def backward_inputs(mp, M, N, K):
    gg = torch.Generator(device="cuda").manual_seed(M + N)
    t = [torch.randn(*s, generator=gg, device="cuda").bfloat16() for s in ((M, N), (M, K), (N, K), (N, K), (M, N), (M, N))]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return t, torch.empty(mp.mpgemm_run_gated_backward_workspace(M, N, K, 1, cus), dtype=torch.uint8, device="cuda")


# Either weight's gradient alone, in tiles of every size and N that ends anywhere in its last tile.
@pytest.mark.parametrize("M,N,K", [(1, 3, 8), (40, 64, 16), (70, 65, 136), (300, 129, 264), (700, 1000, 520), (2048, 2050, 1032), (1500, 4480, 2056)])
def test_backward_of_one_weight(mp, M, N, K):
    t, ws = backward_inputs(mp, M, N, K)
    whole = mp.gemm_gated_backward(*t)
    for want in ((0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1)):
        ws.fill_(0x7F)
        run, out = backward_call(mp, t, want, ws)
        run()
        torch.cuda.synchronize()
        assert all(v is None or torch.equal(v, w) for v, w in zip(out, whole))


# A gradient that is not wanted is not computed either: one weight's takes half of the time of both.
def test_backward_of_one_weight_takes_half(mp):
    t, ws = backward_inputs(mp, 4096, 4096, 4096)
    runs = [backward_call(mp, t, want, ws) for want in ((0, 1, 1), (0, 1, 0), (0, 0, 1))]
    best = [1e9] * 3
    for _ in range(12):
        for i, (run, _) in enumerate(runs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            run()
            a.record()
            for _ in range(3):
                run()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b) / 3)
    print("both, dWg, dWu (ms):", best)
    assert max(best[1:]) < 0.8 * best[0]


# dG = dH U act'(G) and dU = dH act(G) are held in the operands' type. With a gate of 100 (of any activation act' is 1, act is the gate) and
# tokens that are rows of the identity, dWg and dWu show them.
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_fp16_gradients_below_its_normal_numbers(mp, name):
    M = N = 64
    # quarters of the smallest subnormal: every remainder, ties too (numbers of up to 11 bits, so that dH is exact)
    k = (torch.arange(M * N, dtype=torch.float64).reshape(M, N) - 2000).clamp(max=2048)
    dh = (k * 2.0 ** -13).half()
    u = torch.full((M, N), 2.0 ** -13, dtype=torch.float16)
    g = torch.full((M, N), 100.0, dtype=torch.float16)
    x = (1024 * torch.eye(M)).half()
    _, dwg, _ = mp.gemm_gated_backward(dh.cuda(), x.cuda(), None, None, g.cuda(), u.cuda(), act=name, need_dx=False)
    want = (dh.double() * u.double()).half()   # (one rounding of an exact product)
    assert (want != 0).any() and want.abs().max() < 2.0 ** -13
    assert torch.equal(dwg.t().cpu().double(), want.double() * 1024)


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_gradients_past_the_largest_fp16(mp, t):
    dt = lu.TYPES[t]
    M, N, K = 70, 40, 72
    gg = torch.Generator().manual_seed(4)
    x, wg, wu = (torch.rand(*s, generator=gg).to(dt) + 1 for s in ((M, K), (N, K), (N, K)))
    dh, u = (torch.randn(M, N, generator=gg).to(dt) for _ in range(2))
    g = torch.randn(M, N, generator=gg).to(dt)
    dh[33, 7], u[33, 7], g[33, 7] = 400.0, 200.0, 100.0   # dG = 80000, dU = 40000
    want = lu.gated_backward(dh, x, wg, wu, g, u, "silu", torch.bfloat16)
    dx, dwg, dwu = (y.cpu() for y in mp.gemm_gated_backward(*(v.cuda() for v in (dh, x, wg, wu, g, u))))
    if t == "bf16":
        for y, (w, e) in zip((dx, dwg, dwu), want):
            lu.check(y, w, e)
        return
    assert (dx[33] == float("inf")).all() and (dwg[7] == float("inf")).all()
    rest = torch.arange(M) != 33
    assert torch.isfinite(dx[rest]).all() and torch.isfinite(dwg[torch.arange(N) != 7]).all() and torch.isfinite(dwu[torch.arange(N) != 7]).all()


# Every activation in large tiles, in 16 bits and on integers.
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh"])
def test_activations_in_large_tiles(mp, name):
    dt, (M, N, K) = torch.bfloat16, (2100, 1030, 72)
    gg = torch.Generator().manual_seed(9)
    x = torch.randn(M, K, generator=gg).to(dt)
    wg, wu = ((0.3 * torch.randn(N, K, generator=gg)).to(dt) for _ in range(2))
    want, tol = lu.gated(x, wg, wu, name)
    for y, w, e in zip(mp.gemm_gated(x.cuda(), wg.cuda(), wu.cuda(), act=name, keep=True), want, tol):
        lu.check(y, w, lu.rounded_tol(w, e, dt))
    a, b, c = (lu.quantize(v) for v in (x, wg, wu))
    (pg, mg), (pu, mu) = lu.scaled(a, b), lu.scaled(a, c)
    (h, _, _), (e, _, _) = lu.gated_from(pg, pu, 3.01 * 2.0 ** -24 * mg, 3.01 * 2.0 ** -24 * mu, name)
    held = [(q.to(torch.int8).cuda(), s.cuda()) for q, s in (b, c)]
    for t in (torch.float32, dt):
        y = mp.gemm_gated_w8a8(*mp.quantize_i8(x.cuda()), *held[0], *held[1], act=name, dtype=t)
        lu.check(y, h, lu.rounded_tol(h, e, t))
