"""The 8-bit activation checkpoints and the 4-bit group-scale weights: their cases, their plain forms and
what they compute in 64 bits.

Five operators. With `own` true, run() makes the calls that a training or serving program makes of the package;
with `own` false it computes the same thing with elementary torch operations in 32 bits.

  act8     an activation (M x k, bf16) into 8 bits and back: one absmax per 64 features, codes round(127 x / absmax)
  grads    the adapter gradients grad_A, grad_B of a linear layer whose input was kept in 8 bits
  swiglu   y = silu(gate) * up with gate and up kept in 8 bits, and its backward pass from them, which also gives
           y again, in 8 bits (the input of the layer behind it)
  int4     a weight (n x k, bf16) into 4-bit integers with a scale (and a zero point) per group, and back
  linear   h = dequant(W) x for 1 to 16 tokens over such a weight
"""
import math

import torch

own = False

BLOCK = 64  # features that share an absmax


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the attention input of a few sequences' worth of single tokens: what a call costs
        {"name": "act8-16x4096", "op": "act8", "M": 16, "k": 4096},
        # the widest activation of a 7B layer at 2 x 2048 tokens
        {"name": "act8-4096x11008", "op": "act8", "M": 4096, "k": 11008},
        # the tiny layer of the tests
        {"name": "grads-256x256-M8-r4", "op": "grads", "M": 8, "n": 256, "k": 256, "r": 4, "alpha": 8.0},
        # a 7B attention projection at 2 x 2048 tokens
        {"name": "grads-4096x4096-M4096-r16", "op": "grads", "M": 4096, "n": 4096, "k": 4096, "r": 16, "alpha": 32.0},
        # a 70B gate projection at 4096 tokens
        {"name": "grads-28672x8192-M4096-r64", "op": "grads", "M": 4096, "n": 28672, "k": 8192, "r": 64, "alpha": 16.0},
        # the 7B MLP between its projections, a short odd batch
        {"name": "swiglu-77x11008", "op": "swiglu", "M": 77, "n": 11008},
        # the 70B MLP, a ragged long batch
        {"name": "swiglu-2049x28672", "op": "swiglu", "M": 2049, "n": 28672},
        # a merged 7B attention weight made ready for serving
        {"name": "int4-4096x4096-g128", "op": "int4", "n": 4096, "k": 4096, "group": 128, "zero": True},
        # a merged 70B weight, symmetric, short groups
        {"name": "int4-28672x8192-g64", "op": "int4", "n": 28672, "k": 8192, "group": 64, "zero": False},
        # one token through a 7B attention projection: latency
        {"name": "linear-4096x4096-M1-g128", "op": "linear", "M": 1, "n": 4096, "k": 4096, "group": 128, "zero": True},
        # a handful of tokens through a 7B gate projection, symmetric, short groups
        {"name": "linear-11008x4096-M5-g32", "op": "linear", "M": 5, "n": 11008, "k": 4096, "group": 32, "zero": False},
        # 16 sequences' next tokens through a 70B down projection
        {"name": "linear-8192x28672-M16-g128", "op": "linear", "M": 16, "n": 8192, "k": 28672, "group": 128, "zero": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["act8", "grads", "swiglu", "int4", "linear"])
    if op == "act8":
        M, k = _log(rng, 1, 8192), BLOCK * _log(rng, 1, 448)
        return {"op": op, "M": min(M, 4096 * 11008 // k), "k": k}
    if op == "grads":
        M, n, k = _log(rng, 1, 8192), _log(rng, 64, 28672), BLOCK * _log(rng, 1, 448)
        r = rng.choice([1, 4, 8, 13, 16, 32, 64])
        return {"op": op, "M": max(1, min(M, 4096 * (28672 + 8192) // (n + k))), "n": n, "k": k, "r": r, "alpha": float(2 * r)}
    if op == "swiglu":
        M, n = _log(rng, 1, 8192), BLOCK * _log(rng, 1, 448)
        return {"op": op, "M": min(M, 2049 * 28672 // n), "n": n}
    group = rng.choice([32, 64, 128])
    n, k, zero = _log(rng, 16, 28672), 128 * _log(rng, 1, 224), rng.random() < 0.5
    if op == "int4":
        return {"op": op, "n": min(n, 28672 * 8192 // k), "k": k, "group": group, "zero": zero}
    return {"op": op, "M": rng.randint(1, 16), "n": min(n, 8192 * 28672 // k), "k": k, "group": group, "zero": zero}


# ------------------------------------------------------------------------------------------------ inputs

def _normal(shape, std, gen):
    return (torch.randn(shape, device="cuda", generator=gen) * std).bfloat16()


def _activation(M, k, gen):
    """A hidden state: normal, with a few features that are much larger for every token."""
    x = torch.randn(M, k, device="cuda", generator=gen)
    big = torch.rand(k, device="cuda", generator=gen) < 0.003
    return torch.where(big, x * 20.0, x).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "act8":
        s["x"] = _activation(case["M"], case["k"], gen)
    elif op == "grads":
        M, n, k, r = case["M"], case["n"], case["k"], case["r"]
        s["codes"], s["absmax"] = _quantize8(_activation(M, k, gen))
        s["grad_h"] = _normal((M, n), 1.0, gen)
        s["A"], s["B"] = _normal((r, k), 0.01, gen), _normal((n, r), 0.01, gen)
    elif op == "swiglu":
        M, n = case["M"], case["n"]
        s["gate"], s["up"], s["grad_y"] = _normal((M, n), 1.5, gen), _normal((M, n), 1.0, gen), _normal((M, n), 1.0, gen)
    elif op == "int4":
        s["W"] = _normal((case["n"], case["k"]), 0.02, gen)
    else:
        M, n, k, group = case["M"], case["n"], case["k"], case["group"]
        s["x"] = _activation(M, k, gen)
        s["codes"] = torch.randint(0, 256, (n, k // 2), device="cuda", generator=gen, dtype=torch.uint8)
        s["scale"] = (0.004 + 0.004 * torch.rand(n, k // group, device="cuda", generator=gen)).bfloat16()
        s["zero_point"] = None
        if case["zero"]:
            s["zero_point"] = torch.randint(5, 11, (n, k // group), device="cuda", generator=gen, dtype=torch.uint8)
    return s


# ------------------------------------------------------------------------------------------ plain forms

def _quantize8(x):
    """int8 codes (M x k) and the bf16 absmax of each 64 features; halves round away from zero."""
    v = x.float().reshape(x.shape[0], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    # 127 |x| is exact in 32 bits and the quotient of two 8-bit significands is either a half or far from one
    q = torch.floor(v.abs() * 127.0 / torch.where(top > 0, top, 1.0) + 0.5) * torch.sign(v)
    return q.to(torch.int8).reshape(x.shape), top.squeeze(-1).bfloat16()


def _value8(codes, absmax):
    q = codes.float().reshape(codes.shape[0], -1, BLOCK)
    return (q * (absmax.float() / 127.0).unsqueeze(-1)).reshape(codes.shape)


def _value4(codes, scale, zero_point, group):
    n = codes.shape[0]
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(n, -1, group).float()
    z = 8.0 if zero_point is None else zero_point.float().unsqueeze(-1)
    return ((q - z) * scale.float().unsqueeze(-1)).reshape(n, -1)


def _plain(s):
    op = s["op"]
    if op == "act8":
        return _value8(*_quantize8(s["x"])).bfloat16()
    if op == "grads":
        x, gh, f = _value8(s["codes"], s["absmax"]), s["grad_h"].float(), s["alpha"] / s["r"]
        t, u = x @ s["A"].float().t(), gh @ s["B"].float()
        return f * (u.t() @ x), f * (gh.t() @ t)
    if op == "swiglu":
        g, u = s["gate"].float(), s["up"].float()
        y = (g / (1.0 + torch.exp(-g)) * u).bfloat16()
        g, u, gy = _value8(*_quantize8(s["gate"])), _value8(*_quantize8(s["up"])), s["grad_y"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        again = (g * sig * u).bfloat16()
        return (y, (gy * u * sig * (1.0 + g * (1.0 - sig))).bfloat16(), (gy * g * sig).bfloat16(),
                _value8(*_quantize8(again)).bfloat16())
    if op == "int4":
        w = s["W"].float().reshape(s["n"], -1, s["group"])
        if s["zero"]:
            lo, hi = w.amin(-1, keepdim=True).clamp(max=0.0), w.amax(-1, keepdim=True).clamp(min=0.0)
            scale = ((hi - lo) / 15.0).bfloat16().float()
            z = torch.floor(-lo / torch.where(scale > 0, scale, 1.0) + 0.5).clamp(0, 15)
        else:
            scale = (w.abs().amax(-1, keepdim=True) / 7.0).bfloat16().float()
            z = torch.full_like(scale, 8.0)
        q = torch.floor(w.abs() / torch.where(scale > 0, scale, 1.0) + 0.5) * torch.sign(w)
        q = (q + z).clamp(0, 15)
        return ((q - z) * scale).bfloat16().reshape(s["n"], s["k"])
    W = _value4(s["codes"], s["scale"], s["zero_point"], s["group"])
    return (s["x"].float() @ W.t()).bfloat16()


def _own(s):
    import bit_nf4_quantized_25_b200 as q

    op = s["op"]
    if op == "act8":
        return q.act8_dequantize(q.act8_quantize(s["x"]))
    if op == "grads":
        x8 = q.Act8(s["M"], s["k"], s["codes"], s["absmax"])
        return q.qlora_lora_grads_act8(x8, s["grad_h"], s["A"], s["B"], s["alpha"])
    if op == "swiglu":
        y, gate8, up8 = q.swiglu_act8_fwd(s["gate"], s["up"])
        grad_gate, grad_up, y8 = q.swiglu_act8_bwd(gate8, up8, s["grad_y"])
        return y, grad_gate, grad_up, q.act8_dequantize(y8)
    if op == "int4":
        return q.int4_dequantize(q.int4_quantize(s["W"], group=s["group"], zero_point=s["zero"]))
    w = q.Int4Weight(s["n"], s["k"], s["group"], s["codes"], s["scale"], s["zero_point"])
    return q.int4_linear_fwd(w, s["x"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------- from the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def blocks8(x):
        """x to the nearest multiple of absmax / 127 of its 64 features (absmax is one of x's bf16 values)."""
        v = x.double().unflatten(1, (-1, BLOCK))
        m = v.abs().max(dim=-1, keepdim=True).values
        steps = (254.0 * v.abs() + m).div(2.0 * m).floor().copysign(v)
        return torch.where(m == 0, torch.zeros_like(v), steps * m / 127.0).flatten(1)

    if op == "act8":
        return blocks8(s["x"])
    if op == "grads":
        x = (s["codes"].double().unflatten(1, (-1, BLOCK)) * s["absmax"].double()[..., None] / 127.0).flatten(1)
        gh, A, B, scale = s["grad_h"].double(), s["A"].double(), s["B"].double(), case["alpha"] / case["r"]
        return scale * torch.einsum("mj,mk->jk", gh @ B, x), scale * torch.einsum("mn,mj->nj", gh, x @ A.T)
    if op == "swiglu":
        first = s["gate"].double() * torch.sigmoid(s["gate"].double()) * s["up"].double()
        g, u, gy = blocks8(s["gate"]), blocks8(s["up"]), s["grad_y"].double()
        p = torch.sigmoid(g)
        slope = p + g * p * torch.sigmoid(-g)
        return first, gy * u * slope, gy * g * p, blocks8((g * p * u).bfloat16())
    if op == "int4":
        w = s["W"].double().unflatten(1, (-1, case["group"]))
        if case["zero"]:
            bottom = -torch.relu(-w.min(dim=-1, keepdim=True).values)
            step = ((torch.relu(w.max(dim=-1, keepdim=True).values) - bottom) / 15.0).float().bfloat16().double()
            shift = (-bottom / step + 0.5).floor()
        else:
            step = (w.abs().max(dim=-1, keepdim=True).values / 7.0).float().bfloat16().double()
            shift = torch.full_like(step, 8.0)
        level = (w.abs() / step + 0.5).floor().copysign(w)
        level = torch.minimum(torch.maximum(level, -shift), 15.0 - shift)
        return (level * step).flatten(1)
    low, high = s["codes"] % 16, s["codes"].div(16, rounding_mode="floor")
    w = torch.stack([low, high], dim=2).flatten(1).double().unflatten(1, (-1, case["group"]))
    w -= 8.0 if s["zero_point"] is None else s["zero_point"].double()[..., None]
    w *= s["scale"].double()[..., None]
    return s["x"].double() @ w.flatten(1).T


# ------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    eight = 1.0 + 2.0 / BLOCK  # bytes of a kept value
    if op == "act8":  # x read, the values written; the 8-bit form between them written and read
        return {"bytes": case["M"] * case["k"] * (4.0 + 2.0 * eight), "flops": 0.0}
    if op == "grads":
        M, n, k, r = case["M"], case["n"], case["k"], case["r"]
        return {"bytes": M * (k * eight + 2.0 * n) + 6.0 * r * (n + k), "flops": 4.0 * M * r * (n + k)}
    if op == "swiglu":  # forward: gate, up in; y and both in 8 bits out. backward: those and grad_y in; two gradients and y out
        return {"bytes": case["M"] * case["n"] * ((6.0 + 2.0 * eight) + (6.0 + 3.0 * eight) + (2.0 + eight)), "flops": 0.0}
    four = 0.5 + (3.0 if case["zero"] else 2.0) / case["group"]
    if op == "int4":
        return {"bytes": case["n"] * case["k"] * (4.0 + 2.0 * four), "flops": 0.0}
    M, n, k = case["M"], case["n"], case["k"]
    return {"bytes": n * k * four + 2.0 * M * (n + k), "flops": 2.0 * M * n * k}
