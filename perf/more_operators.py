"""Cases of the linear layer in 8-bit integers (a scale for each token and for
each output channel) and of the gated feed-forward block, which is served in
those integers and trained in 16 bits, with the operators' plain forms in
elementary torch operations.

Operators (the "op" of a case):
  quantize    a matrix into 8-bit integers with a scale for each row, and back
  w8a8        Y = (A B^T) sa sb + bias: B is held in integers, A is held too or
              quantised in the call ("dyn")
  gated       H = act(X Wg^T) (X Wu^T), for training with the two products kept
  backward    dX, dWg and dWu of the same from dH and the products that were kept
  gated_w8a8  the gated block with X quantised in the call and weights held in integers

A matrix held in integers is a pair: int8 codes (R x K, a row's largest
magnitude at 127) and R fp32 scales; the value of an element is code times
scale. The held rows start at multiples of 16 bytes.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode batch's activations, quantised once for several projections
        {"name": "quantize 64x4096 f16", "op": "quantize", "M": 64, "K": 4096, "type": "f16"},
        # a weight that is brought into integers
        {"name": "quantize 10240x4096 bf16", "op": "quantize", "M": 10240, "K": 4096, "type": "bf16"},
        # decode of a single token through a 4096 x 4096 layer
        {"name": "w8a8 1x4096x4096 f16", "op": "w8a8", "dyn": True, "M": 1, "N": 4096, "K": 4096, "type": "f16", "bias": False},
        # a decode batch through an 8192-wide layer with a bias
        {"name": "w8a8 16x8192x8192 bf16", "op": "w8a8", "dyn": True, "M": 16, "N": 8192, "K": 8192, "type": "bf16", "bias": True},
        # a prompt of an odd length through a layer of odd sizes
        {"name": "w8a8 333x5000x2100 bf16", "op": "w8a8", "dyn": True, "M": 333, "N": 5000, "K": 2100, "type": "bf16", "bias": True},
        # the largest square product of the benchmark's sweep, both operands held
        {"name": "w8a8 8192x8192x8192 bf16", "op": "w8a8", "dyn": False, "M": 8192, "N": 8192, "K": 8192, "type": "bf16", "bias": False},
        # decode of a single token through the gated block
        {"name": "gated 1x10240x4096 bf16", "op": "gated", "M": 1, "N": 10240, "K": 4096, "type": "bf16", "act": "silu", "keep": False},
        # the forward pass of a training step, 4096 tokens
        {"name": "gated 4096x10240x4096 bf16", "op": "gated", "M": 4096, "N": 10240, "K": 4096, "type": "bf16", "act": "silu", "keep": True},
        # its backward pass
        {"name": "backward 4096x10240x4096 bf16", "op": "backward", "M": 4096, "N": 10240, "K": 4096, "type": "bf16", "act": "silu"},
        # a small ragged layer's backward pass
        {"name": "backward 777x1000x520 f16", "op": "backward", "M": 777, "N": 1000, "K": 520, "type": "f16", "act": "gelu"},
        # a single token, the block served in integers
        {"name": "gated_w8a8 1x10240x4096 bf16", "op": "gated_w8a8", "M": 1, "N": 10240, "K": 4096, "type": "bf16", "act": "silu"},
        # a batch of prompts through it
        {"name": "gated_w8a8 2048x10240x4096 bf16", "op": "gated_w8a8", "M": 2048, "N": 10240, "K": 4096, "type": "bf16", "act": "silu"},
    ]


def _size(rng, lo, hi, odd=0.4):
    """A size spread over the logarithm of [lo, hi], rounded to a multiple of 64 (when it is that large) or left as it falls."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() > odd:
        n = n // 64 * 64
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["quantize", "w8a8", "w8a8", "gated", "gated", "backward", "gated_w8a8"])
    t = rng.choice(["f16", "bf16"])
    if op == "quantize":
        return {"op": op, "M": _size(rng, 1, 10240), "K": _size(rng, 32, 8192), "type": rng.choice(["f16", "bf16", "f32"])}
    # tokens of a decode step or of prompts; a layer's sizes
    m = _size(rng, 1, 64) if op != "backward" and rng.random() < 0.5 else _size(rng, 65, 4096)
    n, k = _size(rng, 64, 10240), _size(rng, 64, 4096)
    if op == "w8a8":
        dyn = rng.random() < 0.7
        return {"op": op, "dyn": dyn, "M": m, "N": n, "K": k, "type": t if dyn else rng.choice(["f16", "bf16", "f32"]), "bias": rng.random() < 0.5}
    case = {"op": op, "M": m, "N": n, "K": k, "type": t, "act": rng.choice(["silu", "gelu", "gelu_tanh"])}
    if op == "gated":
        case["keep"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """Normal rows with a few loud columns, as the inputs of a linear layer have."""
    loud = torch.exp(0.5 * _normal(g, K)).clamp(max=8.0)
    return _normal(g, M, K) * loud


def _store(x):
    """A matrix into codes and scales, as a user's program holds it."""
    code, s = _codes(x)
    M, K = code.shape
    q = torch.zeros((M, (K + 15) // 16 * 16), dtype=torch.int8, device=x.device)
    q[:, :K] = code.to(torch.int8)
    return q[:, :K], s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    state = dict(case)
    t = TYPES[case["type"]]
    if op == "quantize":
        state["x"] = (_activations(g, M, K) if M <= 64 else 0.02 * _normal(g, M, K)).to(t)
        return state
    N = case["N"]
    if op == "w8a8":
        x = _activations(g, M, K).to(t)
        if case["dyn"]:
            state["x"] = x
        else:
            state["a"] = _store(x)
        state["w"] = _store(0.02 * _normal(g, N, K))
        state["bias"] = _normal(g, N).to(t) if case["bias"] else None
        return state
    state["x"] = _activations(g, M, K).to(t)
    if op == "gated_w8a8":
        state["wg"], state["wu"] = _store(0.02 * _normal(g, N, K)), _store(0.02 * _normal(g, N, K))
        return state
    state["wg"], state["wu"] = (0.02 * _normal(g, N, K)).to(t), (0.02 * _normal(g, N, K)).to(t)
    if op == "backward":
        # (gradients in fp16 come with the loss scaled up)
        size = 1.0 if case["type"] == "f16" else 1e-3
        state["dh"] = (size * _normal(g, M, N) * torch.exp(_normal(g, M, 1))).to(t)
        state["g"] = (state["x"].float() @ state["wg"].float().t()).to(t)
        state["u"] = (state["x"].float() @ state["wu"].float().t()).to(t)
    return state


# ---------------------------------------------------------------- plain forms

def _codes(x):
    """Codes (whole numbers in fp32) and fp32 scales of a matrix's rows."""
    s = (x.abs().amax(dim=1).double() / 127).float()
    # (quotients next to a half: in 64 bits)
    q = torch.where(s[:, None] > 0, x.double() / s[:, None].double(), torch.zeros((), dtype=torch.float64, device=x.device))
    return torch.round(q).clamp(-127, 127).float(), s


def _act(name, v):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _slope(name, v):
    if name == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * math.sqrt(0.5 / math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-c * (v + 0.044715 * v * v * v)))
    return s + v * s * (1 - s) * c * (1 + 3 * 0.044715 * v * v)


def _product(a, b):
    """(A B^T) sa sb of two held matrices."""
    return (a[0].float() @ b[0].float().t()) * a[1][:, None] * b[1][None, :]


def run(state):
    op, t = state["op"], TYPES[state["type"]]
    if own:
        import precision_dense_gemm_tiled_amd as mp
        if op == "quantize":
            return mp.dequantize_i8(*mp.quantize_i8(state["x"]), dtype=t)
        if op == "w8a8":
            if state["dyn"]:
                return mp.gemm_w8a8_dyn(state["x"], *state["w"], bias=state["bias"])
            return mp.gemm_w8a8(*state["a"], *state["w"], bias=state["bias"], dtype=t)
        if op == "gated":
            r = mp.gemm_gated(state["x"], state["wg"], state["wu"], act=state["act"], keep=state["keep"])
            return {"h": r[0], "g": r[1], "u": r[2]} if state["keep"] else {"h": r}
        if op == "backward":
            dx, dwg, dwu = mp.gemm_gated_backward(state["dh"], state["x"], state["wg"], state["wu"], state["g"], state["u"], act=state["act"])
            return {"dx": dx, "dwg": dwg, "dwu": dwu}
        return mp.gemm_gated_w8a8_dyn(state["x"], *state["wg"], *state["wu"], act=state["act"])
    if op == "quantize":
        code, s = _codes(state["x"])
        return (code * s[:, None]).to(t)
    if op == "w8a8":
        y = _product(_codes(state["x"]) if state["dyn"] else state["a"], state["w"])
        return (y if state["bias"] is None else y + state["bias"].float()).to(t)
    if op == "gated_w8a8":
        a = _codes(state["x"])
        return (_act(state["act"], _product(a, state["wg"])) * _product(a, state["wu"])).to(t)
    x, wg, wu = state["x"].float(), state["wg"].float(), state["wu"].float()
    if op == "gated":
        g, u = x @ wg.t(), x @ wu.t()
        h = (_act(state["act"], g) * u).to(t)
        return {"h": h, "g": g.to(t), "u": u.to(t)} if state["keep"] else {"h": h}
    dh, g, u = state["dh"].float(), state["g"].float(), state["u"].float()
    dg, du = dh * u * _slope(state["act"], g), dh * _act(state["act"], g)
    return {"dx": (dg @ wg + du @ wu).to(t), "dwg": (dg.t() @ x).to(t), "dwu": (du.t() @ x).to(t)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    size = 4 if case["type"] == "f32" else 2
    if op == "quantize":
        return {"bytes": 2 * M * K * size, "flops": 4 * M * K}
    N = case["N"]
    if op == "w8a8":
        return {"bytes": (M * K * size if case["dyn"] else M * (K + 4)) + N * (K + 4) + M * N * size + (N * size if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "gated_w8a8":
        return {"bytes": M * K * size + 2 * N * (K + 4) + M * N * size, "flops": 4 * M * N * K}
    if op == "gated":
        return {"bytes": (M * K + 2 * N * K + (3 if case["keep"] else 1) * M * N) * size, "flops": 4 * M * N * K}
    return {"bytes": (3 * M * N + 2 * M * K + 4 * N * K) * size, "flops": 8 * M * N * K}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _integers64(x):
    """Integers and scales of rows: the scale is the fp32 number nearest to a 127th of the row's
    largest magnitude, the integer the nearest to the quotient (ties to even)."""
    v = x.double()
    scale = (v.abs().max(dim=1, keepdim=True).values / 127.0).to(torch.float32).double()
    r = v / scale.masked_fill(scale == 0, 1.0)
    low = torch.floor(r)
    up = (r - low > 0.5) | ((r - low == 0.5) & (torch.remainder(low, 2.0) == 1))
    return (low + up.double()).clamp(min=-127.0, max=127.0) * (scale != 0), scale


def _held64(pair):
    return pair[0].double(), pair[1].double().unsqueeze(1)


def _scaled64(a, b):
    return torch.mm(a[0] * a[1], (b[0] * b[1]).t())


def _gate64(name, v):
    """The activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        return v * phi, phi + v * torch.exp(-v.square() / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    th = torch.tanh(k * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th.square()) * k * (1 + 0.134145 * v.square())


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        code, scale = _integers64(state["x"])
        return code * scale
    if op == "w8a8":
        y = _scaled64(_integers64(state["x"]) if case["dyn"] else _held64(state["a"]), _held64(state["w"]))
        return y if state["bias"] is None else y + state["bias"].double()[None, :]
    if op == "gated_w8a8":
        a = _integers64(state["x"])
        return _gate64(case["act"], _scaled64(a, _held64(state["wg"])))[0] * _scaled64(a, _held64(state["wu"]))
    x, wg, wu = (state[k].double() for k in ("x", "wg", "wu"))
    if op == "gated":
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        h = _gate64(case["act"], g)[0] * u
        return {"h": h, "g": g, "u": u} if case["keep"] else {"h": h}
    a, slope = _gate64(case["act"], state["g"].double())
    dh = state["dh"].double()
    dg, du = dh * slope * state["u"].double(), dh * a
    return {"dx": torch.mm(torch.cat([dg, du], dim=1), torch.cat([wg, wu], dim=0)),
            "dwg": torch.mm(dg.t(), x), "dwu": torch.mm(du.t(), x)}
