"""Plain 64-bit 8-bit integer layers and gated blocks on the CPU, for the tests, with the errors that the kernels' roundings allow."""
import math

import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """The smallest subnormal: half of it is what a rounding may take near zero."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def quantize(x):
    """Codes (int64) and scales (fp32) of a CPU matrix's rows, from the definition. (A quotient of two fp32 numbers
    that is not half-way between integers is at least 2^-48 away relative to it, which 64 bits resolve.)"""
    v = x.double()
    bad = ~torch.isfinite(v).all(dim=1)
    clean = torch.where(bad[:, None], torch.zeros_like(v), v)
    s = (clean.abs().amax(dim=1) / 127).float()
    q = torch.where(s[:, None] > 0, clean / s[:, None].double(), torch.zeros_like(v))
    code = torch.round(q).clamp(-127, 127).long()   # torch.round: ties to even
    return code, torch.where(bad, torch.full_like(s, float("nan")), s)


def random_codes(g, rows, K):
    """Every int8 code, -128 too, and scales of several binades."""
    q = torch.randint(-128, 128, (rows, K), generator=g).to(torch.int8)
    s = torch.exp2(torch.randint(-8, 3, (rows,), generator=g).float()) * (1 + torch.rand(rows, generator=g))
    return q, s


def on_gpu(qs, layout="padded"):
    """Codes and scales as a program holds them: rows padded to 16 bytes (the padding holds 85: bytes that no product may use),
    contiguous rows, or rows that start anywhere."""
    q, s = qs
    R, K = q.shape
    if layout == "contiguous":
        return q.contiguous().cuda(), s.cuda()
    ld = (K + 15) // 16 * 16 + (16 if layout == "padded" else 5)
    big = torch.full((R + 1, ld), 85, dtype=torch.int8)
    at = 0 if layout == "padded" else 3
    flat = big.reshape(-1)
    view = flat[at:at + R * ld].reshape(R, ld)
    view[:, :K] = q
    dev = big.cuda().reshape(-1)
    return dev[at:at + R * ld].reshape(R, ld)[:, :K], s.cuda()


def rows_on_gpu(x, layout="contiguous"):
    """A matrix with contiguous rows, padded ones (NaN in the padding), or rows that start anywhere."""
    R, K = x.shape
    if layout == "contiguous":
        return x.contiguous().cuda()
    ld = (K + 7) // 8 * 8 + (8 if layout == "padded" else 3)
    big = torch.full(((R + 1) * ld,), float("nan"), dtype=x.dtype)
    at = 0 if layout == "padded" else 1
    big[at:at + R * ld].reshape(R, ld)[:, :K] = x
    return big.cuda()[at:at + R * ld].reshape(R, ld)[:, :K]


def scaled(a, b, bias=None):
    """The product of two held matrices, and its terms' magnitude, in 64 bits."""
    p = (a[0].double() @ b[0].double().t()) * a[1].double()[:, None] * b[1].double()[None, :]
    y = p if bias is None else p + bias.double()[None, :]
    return y, p.abs() + (0 if bias is None else bias.double().abs()[None, :])


def scaled_tol(y, mag, dtype):
    """One rounding to the type (half a step), after four in fp32 (the sum, two scales, the bias) of half a step
    of 2^-23 each on at most `mag`, the later ones on what the earlier left."""
    return half_step(dtype) * y.abs() * (1 + 2.0 ** -20) + 4.01 * 2.0 ** -24 * mag + smallest(dtype)


def act(name, v):
    """The activation and its derivative in 64 bits."""
    v = v.double()
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    if name == "gelu":
        phi = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * phi, phi + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * k * (1 + 3 * 0.044715 * v * v)


# Any of the three has a slope of at most 1.13. Its evaluation in fp32: the exponential's argument is off by a few
# 2^-24 of itself, which the exponential's decay keeps at a few 2^-23 of the sigmoid times |v|.
LIPSCHITZ, ACT_ERR = 1.13, 8 * 2.0 ** -23
# The derivative's factor v (1 - s) s multiplies the rounding of 1 - s, 2^-23, by at most 35 (gelu_tanh at |v| = 5, past which 1 - s is 0).
SLOPE_ERR = 64 * 2.0 ** -23


def sum_err(t, K):
    """fp32 sums of K products of 16-bit numbers with magnitudes that sum to t: a matrix instruction adds its 32 products in at
    most 8 steps, each off by at most 2^-23 of the magnitudes so far, and up to 24 partial results are joined."""
    return (K / 4 + 24) * 2.0 ** -23 * t


def gated(x, wg, wu, name):
    """H, G, U and the tolerances of H, G and U before their rounding to the type."""
    xd, gd, ud = x.double(), wg.double(), wu.double()
    g, u = xd @ gd.t(), xd @ ud.t()
    K = x.shape[1]
    dg, du = sum_err(xd.abs() @ gd.abs().t(), K), sum_err(xd.abs() @ ud.abs().t(), K)
    return gated_from(g, u, dg, du, name)


def gated_from(g, u, dg, du, name):
    a = act(name, g)[0]
    da = LIPSCHITZ * dg + ACT_ERR * (g.abs() + dg)
    h = a * u
    dh = (u.abs() + du) * da + a.abs() * du + 2.0 ** -23 * h.abs()
    return (h, g, u), (dh, dg, du)


def rounded_tol(y, d, dtype):
    """One rounding of a value that is off by at most d."""
    return d + half_step(dtype) * (y.abs() + d) + smallest(dtype)


def gated_backward(dh, x, wg, wu, g, u, name, dtype):
    """dX, dWg, dWu in 64 bits and their tolerances: dG and dU are rounded to the type once (half a step), after their evaluation in
    fp32; the sums and the final rounding come on top."""
    a, slope = act(name, g)
    dhd, ud = dh.double(), u.double()
    dg, du = dhd * ud * slope, dhd * a
    eg = (dhd * ud).abs() * SLOPE_ERR + dg.abs() * 2.0 ** -22
    eu = dhd.abs() * (ACT_ERR * g.double().abs()) + du.abs() * 2.0 ** -23
    eg = rounded_tol(dg, eg, dtype)
    eu = rounded_tol(du, eu, dtype)
    xd, gd, wd = x.double(), wg.double(), wu.double()
    M, N = dh.shape
    dx = dg @ gd + du @ wd
    tx = eg @ gd.abs() + eu @ wd.abs()
    tx = tx + sum_err(dg.abs() @ gd.abs() + du.abs() @ wd.abs() + tx, 2 * N)
    out = [(dx, rounded_tol(dx, tx, dtype))]
    for d, e in ((dg, eg), (du, eu)):
        y = d.t() @ xd
        t = e.t() @ xd.abs()
        t = t + sum_err(d.abs().t() @ xd.abs() + t, M)
        out.append((y, rounded_tol(y, t, dtype)))
    return out


def check(got, y, tol):
    got = got.double().cpu()
    nan = torch.isnan(y)
    assert got.shape == y.shape
    assert torch.equal(torch.isnan(got), nan)
    off = (got - y).abs()
    over = (off > tol) & ~nan
    assert not over.any(), f"{int(over.sum())} outputs off, first at {over.nonzero()[0].tolist()}: " \
                           f"{got[over][0].item()} for {y[over][0].item()} +- {tol[over][0].item()}"
