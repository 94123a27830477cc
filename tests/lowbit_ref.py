"""Plain 64-bit forms of the 8-bit activations, the SwiGLU over them and the 4-bit integer weights,
written from their definitions; the tests compare the kernels with these."""
import numpy as np
import torch

HALF_STEP = 2.0 ** -8  # bf16: half a step relative to the value


def act8(x: torch.Tensor):
    """(codes as float64, absmax as float64) of x; halves away from zero; NaN blocks as the format says."""
    v = x.double().reshape(x.shape[0], -1, 64)
    a = v.abs().amax(-1, keepdim=True)
    a = torch.where(torch.isfinite(v).all(-1, keepdim=True), a, torch.full_like(a, float("nan")))
    q = torch.floor((254.0 * v.abs() + a) / (2.0 * a)) * torch.sign(v)
    q = torch.where((a > 0).expand_as(q), q, torch.zeros_like(q))
    return q.reshape(x.shape), a.squeeze(-1)


def act8_values(codes: torch.Tensor, absmax: torch.Tensor) -> torch.Tensor:
    q = codes.double().reshape(codes.shape[0], -1, 64)
    return (q * (absmax.double() / 127.0).unsqueeze(-1)).reshape(codes.shape)


def swiglu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def swiglu_grads(g, u, dy):
    s = 1.0 / (1.0 + torch.exp(-g))
    return dy * u * (s + g * s * (1.0 - s)), dy * g * s


def int4(W: torch.Tensor, group: int, zero_point: bool):
    """(codes, scale, zero points) of W: the scale in fp32 and bf16 as the format says, the codes in 64 bits."""
    w = W.float().cpu().numpy().reshape(W.shape[0], -1, group)
    zero = np.float32(0.0)
    if zero_point:
        lo, hi = np.minimum(w.min(-1), zero), np.maximum(w.max(-1), zero)
        span = (hi - lo) / np.float32(15.0)
    else:
        lo, span = None, np.abs(w).max(-1) / np.float32(7.0)
    assert span.dtype == np.float32
    scale = torch.from_numpy(span).bfloat16()
    s = scale.double().numpy()
    safe = np.where(s > 0, s, 1.0)
    if zero_point:
        z = np.clip(np.floor(-lo.astype(np.float64) / safe + 0.5), 0, 15) * (s > 0)
    else:
        z = np.full(s.shape, 8.0)
    d = w.astype(np.float64)
    q = np.floor(np.abs(d) / safe[..., None] + 0.5) * np.sign(d) * (s > 0)[..., None]
    q = np.clip(q + z[..., None], 0, 15)
    return q.reshape(W.shape).astype(np.int64), scale, z.astype(np.int64)


def int4_unpack(codes: torch.Tensor) -> torch.Tensor:
    return torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)


def int4_values(codes: torch.Tensor, scale: torch.Tensor, zero_point, group: int) -> torch.Tensor:
    q = int4_unpack(codes).double().reshape(codes.shape[0], -1, group)
    z = 8.0 if zero_point is None else zero_point.double().unsqueeze(-1)
    return ((q - z) * scale.double().unsqueeze(-1)).reshape(codes.shape[0], -1)


def lora_grads(x, gh, A, B, s):
    """(grad_A, grad_B, bounds of both) in 64 bits; the bounds are sums of the sizes of all terms, in units of
    which the fp32 arithmetic errs."""
    t, u = x @ A.t(), gh @ B
    tb, ub = x.abs() @ A.abs().t(), gh.abs() @ B.abs()
    return s * (u.t() @ x), s * (gh.t() @ t), s * (ub.t() @ x.abs()), s * (gh.abs().t() @ tb)
