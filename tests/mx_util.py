"""Plain 64-bit MXFP4 and Newton-Schulz on the CPU, for the tests."""
import numpy as np
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def quantize(x):
    """Codes (M x 16 nb uint8) and scales (M x nb uint8) of a CPU matrix, from the definition: the nearest grid
    value, ties to the one with an even code."""
    M, K = x.shape
    nb = (K + 31) // 32
    v = torch.zeros((M, nb * 32), dtype=torch.float64)
    v[:, :K] = x.double()
    v = v.reshape(M, nb, 32)
    amax = v.abs().amax(dim=2)
    bad = ~torch.isfinite(v).all(dim=2)
    safe = torch.where(bad | (amax == 0), torch.ones_like(amax), amax)
    b = (torch.frexp(safe)[1] - 1 - 2 + 127).clamp(0, 254)   # frexp: amax = m 2^e with m in [1/2, 1)
    b = torch.where(amax == 0, torch.zeros_like(b), b)
    b = torch.where(bad, torch.full_like(b, 255), b)
    r = torch.where(bad[:, :, None], torch.zeros_like(v), v).abs() / torch.exp2(b.double().clamp(max=254) - 127)[:, :, None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    code = torch.zeros(r.shape, dtype=torch.int64)
    for i in range(7):   # past the middle, or on it with an even upper code
        code += ((r > mid[i]) | ((r == mid[i]) & (i % 2 == 1))).long()
    code = torch.where(torch.signbit(v) & ~bad[:, :, None], code + 8, code).reshape(M, nb * 32)
    q = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    return q, b.to(torch.uint8)


def values(q, s, K):
    """The 64-bit values of codes and scales."""
    code = torch.stack([q & 15, q >> 4], dim=2).reshape(q.shape[0], -1).long()
    v = GRID[code & 7] * torch.where(code >= 8, -1.0, 1.0).double()
    scale = torch.exp2(s.double() - 127)
    scale = torch.where(s == 255, torch.full_like(scale, float("nan")), scale)
    return (v.reshape(q.shape[0], -1, 32) * scale[:, :, None]).reshape(q.shape[0], -1)[:, :K]


def on_gpu(qs):
    """Codes and scales as a program holds them: scale rows padded to 16 bytes (the padding is 255: NaN scales that
    no product may use)."""
    q, s = qs
    pad = torch.full((s.shape[0], (s.shape[1] + 15) // 16 * 16), 255, dtype=torch.uint8)
    pad[:, :s.shape[1]] = s
    return q.contiguous().cuda(), pad.cuda()[:, :s.shape[1]]


def random_held(g, rows, K, spread=3):
    """A random MXFP4 matrix: every code, scales 2^-spread ... 2^spread."""
    nb = (K + 31) // 32
    q = torch.randint(0, 256, (rows, 16 * nb), generator=g, dtype=torch.uint8)
    code = torch.stack([q & 15, q >> 4], dim=2).reshape(rows, -1)
    code[:, K:] = 0
    q = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    s = torch.randint(127 - spread, 128 + spread, (rows, nb), generator=g).to(torch.uint8)
    return q, s


def gemm_tol(y, t, nb, dtype):
    """One rounding to the result's type (half a step), and fp32 sums: each block of 32 products is added with at
    most a step of 2^-23 of the magnitudes so far (t: the sum of the products' magnitudes), and up to 24 partial
    results are joined."""
    return half_step(dtype) * y.abs() + (nb + 24) * 2.0 ** -23 * t + torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def check(got, y, tol):
    got = got.double().cpu()
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan)
    off = (got - y).abs()
    over = (off > tol) & ~nan
    assert not over.any(), f"{int(over.sum())} outputs off, first at {over.nonzero()[0].tolist()}: " \
                           f"{got[over][0].item()} for {y[over][0].item()}"


def newton_schulz(x, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """64-bit orthogonalisation of one CPU matrix."""
    a, b, c = coeffs
    u = x.double()
    u = u / (torch.linalg.vector_norm(u) + eps)
    flip = u.shape[0] > u.shape[1]
    u = u.t() if flip else u
    for _ in range(steps):
        A = u @ u.t()
        u = a * u + (b * A + c * (A @ A)) @ u
    return u.t() if flip else u


def bits(t):
    return np.asarray(t.cpu())
