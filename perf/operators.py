"""Cases of the 4-bit floating-point linear layer (MXFP4: e2m1 elements, one
e8m0 scale per 32 of the contracted axis) and of the orthogonalised update of
its weight, with the operators' plain forms in elementary torch operations.

Operators (the "op" of a case):
  quantize   a matrix into MXFP4 in both orientations, as a weight is after an
             update (the product needs W, its backward pass W^T), and back
  dyn        Y = MX(X) W^T + bias: X is quantised in the call, W is held in MXFP4
  gemm       Y = A B^T with both operands held in MXFP4
  backward   dX = MX(dY) W, dW = MX(dY^T) X: gradients of a linear layer whose
             W^T and X^T are held in MXFP4
  ortho      Newton-Schulz orthogonalisation of a batch of gradient matrices

An MXFP4 matrix is a pair of uint8 tensors: codes, rows of 16 bytes per block
of 32 (low nibble = even element, zero past the row's end), and scales, one
byte per block.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


def listed():
    return [
        # one decoded token's activations of a 4096-wide layer: latency
        {"name": "quantize 1x4096 f16", "op": "quantize", "M": 1, "K": 4096, "type": "f16"},
        # a 4096 x 4096 weight after its update
        {"name": "quantize 4096x4096 bf16", "op": "quantize", "M": 4096, "K": 4096, "type": "bf16"},
        # decode of a single token through a 4096 x 4096 layer
        {"name": "dyn 1x4096x4096 f16", "op": "dyn", "M": 1, "N": 4096, "K": 4096, "type": "f16", "bias": False},
        # a decode batch through an 8192-wide layer with a bias
        {"name": "dyn 16x8192x8192 bf16", "op": "dyn", "M": 16, "N": 8192, "K": 8192, "type": "bf16", "bias": True},
        # a prompt of an odd length through a layer of odd sizes
        {"name": "dyn 333x5000x2100 bf16", "op": "dyn", "M": 333, "N": 5000, "K": 2100, "type": "bf16", "bias": True},
        # a batch of prompts through a 4096 x 4096 layer
        {"name": "dyn 2048x4096x4096 bf16", "op": "dyn", "M": 2048, "N": 4096, "K": 4096, "type": "bf16", "bias": False},
        # the largest square product of the benchmark's sweep
        {"name": "gemm 8192x8192x8192 bf16", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "type": "bf16"},
        # a small product, fp32 result
        {"name": "gemm 512x512x512 f32", "op": "gemm", "M": 512, "N": 512, "K": 512, "type": "f32"},
        # a training step's gradients: 4096 tokens, 4096 x 4096 weight
        {"name": "backward 4096x4096x4096", "op": "backward", "M": 4096, "N": 4096, "K": 4096, "type": "bf16"},
        # the same with an odd number of tokens and a ragged layer
        {"name": "backward 777x1000x520", "op": "backward", "M": 777, "N": 1000, "K": 520, "type": "f16"},
        # the square projections of twelve small layers, updated together
        {"name": "ortho 12x512x512 bf16", "op": "ortho", "batch": 12, "M": 512, "N": 512, "type": "bf16"},
        # one large rectangular weight, taller than wide
        {"name": "ortho 1x8192x2048 bf16", "op": "ortho", "batch": 1, "M": 8192, "N": 2048, "type": "bf16"},
    ]


def _size(rng, lo, hi, odd=0.4):
    """A size spread over the logarithm of [lo, hi], rounded to a multiple of 64 (when it is that large) or left as it falls."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() > odd:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["quantize", "dyn", "dyn", "gemm", "backward", "ortho"])
    t = rng.choice(["f16", "bf16"])
    if op == "quantize":
        return {"op": op, "M": _size(rng, 1, 8192), "K": _size(rng, 32, 8192), "type": rng.choice(["f16", "bf16", "f32"])}
    if op == "dyn":
        m = _size(rng, 1, 64) if rng.random() < 0.5 else _size(rng, 65, 4096)
        return {"op": op, "M": m, "N": _size(rng, 64, 8192), "K": _size(rng, 64, 8192), "type": t, "bias": rng.random() < 0.5}
    if op == "gemm":
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 8192), "K": _size(rng, 64, 8192), "type": rng.choice(["f16", "bf16", "f32"])}
    if op == "backward":
        return {"op": op, "M": _size(rng, 64, 4096), "N": _size(rng, 64, 4096), "K": _size(rng, 64, 4096), "type": t}
    m, n = _size(rng, 64, 4096), _size(rng, 64, 4096)
    most = max(1, min(16, (1 << 23) // (m * n)))
    return {"op": op, "batch": rng.randint(1, most), "M": m, "N": n, "type": t}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """Normal rows with a few loud columns, as the inputs of a linear layer have."""
    loud = torch.exp(1.0 * _normal(g, K)).clamp(max=20.0)
    return _normal(g, M, K) * loud


def _gradients(g, M, N):
    """Small values whose size differs from token to token."""
    return 1e-3 * _normal(g, M, N) * torch.exp(_normal(g, M, 1))


def _store(x):
    """A matrix into MXFP4 codes and scale bytes, as a user's program holds it."""
    code, e = _codes(x)
    M, nb = e.shape
    c = code.to(torch.uint8)
    q = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
    s = torch.zeros((M, (nb + 15) // 16 * 16), dtype=torch.uint8, device=x.device)
    s[:, :nb] = (e + 127).to(torch.uint8)
    return q, s[:, :nb]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M = case["op"], case["M"]
    state = dict(case)
    t = TYPES[case["type"]]
    if op == "quantize":
        state["x"] = (_activations(g, M, case["K"]) if M < 64 else 0.02 * _normal(g, M, case["K"])).to(t)
    elif op == "dyn":
        N, K = case["N"], case["K"]
        state["x"] = _activations(g, M, K).to(t)
        state["w"] = _store(0.02 * _normal(g, N, K))
        state["bias"] = _normal(g, N).to(t) if case["bias"] else None
    elif op == "gemm":
        state["a"] = _store(_activations(g, M, case["K"]))
        state["b"] = _store(0.02 * _normal(g, case["N"], case["K"]))
    elif op == "backward":
        N, K = case["N"], case["K"]
        state["dy"] = _gradients(g, M, N).to(t)
        state["wt"] = _store((0.02 * _normal(g, N, K)).t().contiguous())
        state["xt"] = _store(_activations(g, M, K).t().contiguous())
    else:
        B, N = case["batch"], case["N"]
        m = min(M, N, 64)
        low = _normal(g, B, M, m) @ (_normal(g, B, m, N) / torch.arange(1, m + 1, device="cuda", dtype=torch.float32)[:, None])
        state["g"] = (1e-3 * (low + _normal(g, B, M, N))).to(t)
    return state


# ---------------------------------------------------------------- plain forms

def _codes(x):
    """e2m1 codes (M x 32 nb, zero past the row's end) and exponents (M x nb) of fp32 rows."""
    M, K = x.shape
    nb = (K + 31) // 32
    v = torch.zeros((M, nb * 32), dtype=torch.float32, device=x.device)
    v[:, :K] = x
    v = v.reshape(M, nb, 32)
    amax = v.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax)[1].to(torch.int32) - 3, torch.full_like(amax, -127, dtype=torch.int32)).clamp(-127, 127)
    r = torch.ldexp(v.abs(), -e[:, :, None])
    code = ((r > 0.25).to(torch.int32) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = code + 8 * torch.signbit(v)
    return code.reshape(M, nb * 32), e


def _values_of(code, e):
    """fp32 values of codes and exponents."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    mag = table[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0)
    M, nb = e.shape
    return torch.ldexp(mag.reshape(M, nb, 32), e[:, :, None]).reshape(M, nb * 32)


def _rounded(x):
    """fp32 matrix -> the values of its MXFP4 form."""
    return _values_of(*_codes(x.float()))[:, :x.shape[1]]


def _held(qs, K):
    """The values that a held MXFP4 matrix stands for."""
    q, s = qs
    code = torch.stack([q & 15, q >> 4], dim=2).reshape(q.shape[0], -1).to(torch.int32)
    return _values_of(code, s.to(torch.int32) - 127)[:, :K]


def _orthogonal(x):
    a, b, c = COEFFS
    x = x.float()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    for _ in range(STEPS):
        A = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.transpose(1, 2).contiguous() if tall else x


def run(state):
    op, t = state["op"], TYPES[state["type"]]
    if own:
        import precision_dense_gemm_tiled_amd as mp
        if op == "quantize":
            x = state["x"]
            q, s, qt, st = mp.quantize_mxfp4_both(x)
            return {"rows": mp.dequantize_mxfp4(q, s, x.shape[1], torch.bfloat16),
                    "columns": mp.dequantize_mxfp4(qt, st, x.shape[0], torch.bfloat16)}
        if op == "dyn":
            return mp.gemm_mxfp4_dyn(state["x"], *state["w"], bias=state["bias"])
        if op == "gemm":
            return mp.gemm_mxfp4(*state["a"], *state["b"], state["K"], dtype=t)
        if op == "backward":
            dx, dw = mp.gemm_mxfp4_backward(state["dy"], *state["wt"], *state["xt"])
            return {"dx": dx, "dw": dw}
        return mp.newton_schulz(state["g"], steps=STEPS, coeffs=COEFFS, eps=EPS)
    if op == "quantize":
        x = state["x"]
        return {"rows": _rounded(x).to(torch.bfloat16), "columns": _rounded(x.t()).to(torch.bfloat16)}
    if op == "dyn":
        y = _rounded(state["x"]) @ _held(state["w"], state["K"]).t()
        return (y if state["bias"] is None else y + state["bias"].float()).to(t)
    if op == "gemm":
        return (_held(state["a"], state["K"]) @ _held(state["b"], state["K"]).t()).to(t)
    if op == "backward":
        dy = state["dy"]
        dx = _rounded(dy) @ _held(state["wt"], state["N"]).t()
        dw = _rounded(dy.t()) @ _held(state["xt"], state["M"]).t()
        return {"dx": dx.to(t), "dw": dw}
    return _orthogonal(state["g"]).to(t)


# ---------------------------------------------------------------- what a pass cannot do without

def _mx_bytes(rows, cols):
    """Codes and scales of an MXFP4 matrix."""
    return rows * (-(-cols // 32)) * 17


def work(case):
    op, M = case["op"], case["M"]
    size = 4 if case["type"] == "f32" else 2
    if op == "quantize":
        K = case["K"]
        return {"bytes": M * K * size + 2 * M * K * 2, "flops": 4 * M * K}
    N = case["N"]
    if op == "ortho":
        m, n = min(M, N), max(M, N)
        return {"bytes": 2 * case["batch"] * M * N * size, "flops": case["batch"] * STEPS * (3 * m * m * n + m * m * m)}
    K = case["K"]
    if op == "dyn":
        return {"bytes": M * K * size + _mx_bytes(N, K) + M * N * size + (N * size if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "gemm":
        return {"bytes": _mx_bytes(M, K) + _mx_bytes(N, K) + M * N * size, "flops": 2 * M * N * K}
    return {"bytes": M * N * size + _mx_bytes(K, N) + _mx_bytes(K, M) + M * K * size + N * K * 4, "flops": 4 * M * N * K}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _blocks64(x):
    """Each element of a matrix as MXFP4 holds it, in 64 bits: the scale is the power of two two binades
    under the block's largest magnitude, the element the nearest of the e2m1 grid (ties to even)."""
    x = x.double()
    M, K = x.shape
    pad = (-K) % 32
    v = torch.cat([x, x.new_zeros((M, pad))], dim=1).reshape(M, -1, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2).clamp(-127, 127))
    u = v / scale
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=1.0, max=7.99)))) / 2
    r = (torch.round(u / step) * step).clamp(-6.0, 6.0)
    return (r * scale).reshape(M, -1)[:, :K]


def _decode64(qs, K):
    q, s = qs
    q = q.long()
    n = torch.stack((q % 16, q // 16), dim=-1).flatten(1)
    sign, ex, man = 1 - 2 * (n // 8).double(), (n // 2) % 4, n % 2
    mag = torch.where(ex == 0, 0.5 * man.double(), torch.exp2(ex.double() - 1) * (1 + 0.5 * man.double()))
    return ((sign * mag).reshape(q.shape[0], -1, 32) * torch.exp2(s.double() - 127)[:, :, None]).flatten(1)[:, :K]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"rows": _blocks64(state["x"]), "columns": _blocks64(state["x"].t())}
    if op == "dyn":
        y = torch.mm(_blocks64(state["x"]), _decode64(state["w"], case["K"]).t())
        return y if state["bias"] is None else y + state["bias"].double()[None, :]
    if op == "gemm":
        return torch.mm(_decode64(state["a"], case["K"]), _decode64(state["b"], case["K"]).t())
    if op == "backward":
        dy = state["dy"]
        return {"dx": torch.mm(_blocks64(dy), _decode64(state["wt"], case["N"]).t()),
                "dw": torch.mm(_blocks64(dy.t()), _decode64(state["xt"], case["M"]).t())}
    k1, k3, k5 = COEFFS
    found = []
    for m in state["g"].double().unbind(0):
        u = m / (torch.linalg.vector_norm(m) + EPS)
        flip = u.shape[0] > u.shape[1]
        if flip:
            u = u.t()
        for _ in range(STEPS):
            gram = torch.mm(u, u.t())
            u = k1 * u + torch.mm(k3 * gram + k5 * torch.mm(gram, gram), u)
        found.append(u.t() if flip else u)
    return torch.stack(found)
