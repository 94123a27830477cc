"""Thin Python binding of ``libqlora_nf4.so`` (the C ABI in ``include/qlora_nf4.h``).

Argument marshalling only: torch tensors supply device memory and the current CUDA
stream; every step of the computation runs in the library's sm_100a kernels. There is
no fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import importlib.util
import os
import threading
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlora_nf4.so")

QN_OK, QN_EINVAL, QN_ESHAPE, QN_EALIGN, QN_ECUDA, QN_EWORKSPACE, QN_ETIMEOUT = range(7)
BLOCK, GROUP, MAX_RANK = 64, 256, 256
QUANT_TYPES = {"nf4": 0, "fp4": 1}  # QN_QUANT_NF4, QN_QUANT_FP4
CONST_DQ, CONST_F32 = 0, 1           # QN_CONST_DQ, QN_CONST_F32

EXPORTED = ("qn_nf4_sizes", "qn_weight_sizes", "qn_quantize_workspace_size", "nf4_quantize", "nf4_quantize_static_ws", "nf4_dequantize",
            "qlora_workspace_size", "qlora_workspace_check", "qlora_linear_fwd", "qlora_linear_bwd_x",
            "qlora_merge_bf16", "qlora_lora_grads_workspace_size", "qlora_lora_grads", "qlora_linear_fwd_dropout",
            "qlora_linear_bwd_x_dropout", "qlora_lora_grads_dropout", "qn_act8_sizes", "act8_quantize",
            "act8_dequantize", "qlora_lora_grads_act8_workspace_size", "qlora_lora_grads_act8", "swiglu_act8_fwd",
            "swiglu_act8_bwd", "qn_int4_sizes", "int4_quantize", "int4_dequantize", "int4_linear_fwd",
            "qn_status_string",
            "qn_last_error", "qn_launch_count", "qn_selftest_wait_timeout", "qn_selftest_grads_give_up")


class QNError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class CWeight(ctypes.Structure):
    """qn_nf4_weight (see the header); fields left at zero mean NF4 with double quantisation."""
    _fields_ = [("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("absmax_q", ctypes.c_void_p), ("group_scale", ctypes.c_void_p),
                ("absmax_mean", ctypes.c_void_p), ("quant_type", ctypes.c_int32), ("const_format", ctypes.c_int32),
                ("absmax", ctypes.c_void_p)]


class CDropout(ctypes.Structure):
    """qn_lora_dropout (see the header): rate p, generator key and element-index offset."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class CAct8(ctypes.Structure):
    """qn_act8 (see the header)."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("absmax", ctypes.c_void_p)]


class CInt4(ctypes.Structure):
    """qn_int4_weight (see the header); zero_point None means 8 for every group."""
    _fields_ = [("n_out", ctypes.c_int64), ("k_in", ctypes.c_int64), ("group", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero_point", ctypes.c_void_p)]


def _dropout_struct(dropout) -> CDropout:
    p, seed, offset = dropout
    return CDropout(float(p), int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFFFFFFFFFF)


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load the library (once). Raises if it is missing: there is no other path."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m bit_nf4_quantized_25_b200.build`")
        lib = ctypes.CDLL(p)
        P, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
        W = ctypes.POINTER(CWeight)
        st = ctypes.c_int
        lib.qn_nf4_sizes.argtypes = [i64, i64, sz, sz, sz, sz]
        lib.qn_weight_sizes.argtypes = [i64, i64, ctypes.c_int, sz, sz, sz, sz, sz]
        lib.qn_quantize_workspace_size.argtypes = [i64, i64, sz]
        lib.nf4_quantize.argtypes = [P, W, P, ctypes.c_size_t, P]
        lib.nf4_dequantize.argtypes = [W, P, P]
        lib.nf4_quantize_static_ws.argtypes = [P, W, P]
        lib.qlora_workspace_size.argtypes = [i64, i64, i64, ctypes.c_int, sz]
        lib.qlora_workspace_check.argtypes = [P, P]
        lib.qn_selftest_wait_timeout.argtypes = [P, ctypes.c_size_t, P]
        lib.qlora_linear_fwd.argtypes = [W, P, i64, P, P, ctypes.c_int, ctypes.c_float, P, P, ctypes.c_size_t, P]
        lib.qlora_linear_bwd_x.argtypes = lib.qlora_linear_fwd.argtypes
        lib.qlora_merge_bf16.argtypes = [W, P, P, ctypes.c_int, ctypes.c_float, P, P]
        lib.qlora_lora_grads_workspace_size.argtypes = [i64, ctypes.c_int, sz]
        lib.qlora_lora_grads.argtypes = [P, P, i64, i64, i64, P, P, ctypes.c_int, ctypes.c_float, P, P, P,
                                         ctypes.c_size_t, P]
        D = ctypes.POINTER(CDropout)
        lib.qlora_linear_fwd_dropout.argtypes = [W, P, i64, P, P, ctypes.c_int, ctypes.c_float, D, P, P,
                                                 ctypes.c_size_t, P]
        lib.qlora_linear_bwd_x_dropout.argtypes = lib.qlora_linear_fwd_dropout.argtypes
        lib.qlora_lora_grads_dropout.argtypes = [P, P, i64, i64, i64, P, P, ctypes.c_int, ctypes.c_float, D, P, P,
                                                 P, ctypes.c_size_t, P]
        A8, I4 = ctypes.POINTER(CAct8), ctypes.POINTER(CInt4)
        lib.qn_act8_sizes.argtypes = [i64, i64, sz, sz]
        lib.act8_quantize.argtypes = [P, A8, P]
        lib.act8_dequantize.argtypes = [A8, P, P]
        lib.qlora_lora_grads_act8_workspace_size.argtypes = [i64, i64, ctypes.c_int, sz]
        lib.qlora_lora_grads_act8.argtypes = [A8, P, i64, P, P, ctypes.c_int, ctypes.c_float, D, P, P, P,
                                              ctypes.c_size_t, P]
        lib.swiglu_act8_fwd.argtypes = [P, P, P, A8, A8, P]
        lib.swiglu_act8_bwd.argtypes = [A8, A8, P, P, P, A8, P]
        lib.qn_int4_sizes.argtypes = [i64, i64, ctypes.c_int, sz, sz, sz]
        lib.int4_quantize.argtypes = [P, I4, P]
        lib.int4_dequantize.argtypes = [I4, P, P]
        lib.int4_linear_fwd.argtypes = [I4, P, i64, P, P]
        lib.qn_selftest_grads_give_up.argtypes = lib.qlora_lora_grads_act8.argtypes
        for f in ("qlora_lora_grads_act8_workspace_size", "qlora_lora_grads_act8", "qn_selftest_grads_give_up", "qn_act8_sizes", "act8_quantize",
                  "act8_dequantize", "swiglu_act8_fwd", "swiglu_act8_bwd", "qn_int4_sizes", "int4_quantize",
                  "int4_dequantize", "int4_linear_fwd"):
            getattr(lib, f).restype = st
        for f in ("qlora_merge_bf16", "qlora_lora_grads_workspace_size", "qlora_lora_grads", "qn_nf4_sizes", "qn_quantize_workspace_size", "nf4_quantize", "nf4_quantize_static_ws", "nf4_dequantize",
                  "qlora_workspace_size", "qlora_workspace_check", "qlora_linear_fwd", "qlora_linear_bwd_x",
                  "qlora_linear_fwd_dropout", "qlora_linear_bwd_x_dropout", "qlora_lora_grads_dropout"):
            getattr(lib, f).restype = st
        lib.qn_status_string.argtypes = [st]
        lib.qn_status_string.restype = ctypes.c_char_p
        lib.qn_last_error.restype = ctypes.c_char_p
        lib.qn_launch_count.argtypes = [ctypes.c_int]
        lib.qn_launch_count.restype = ctypes.c_uint64
        if path is None:
            _lib = lib
        return lib


def _check(status: int, what: str):
    if status != QN_OK:
        lib = load()
        raise QNError(status, f"{what}: {lib.qn_status_string(status).decode()} ({lib.qn_last_error().decode()})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev_bf16(t: torch.Tensor, name: str):
    if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")


def _expect_shape(t: torch.Tensor, shape, name: str):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def check_linear_shapes(n_out: int, k_in: int, act: torch.Tensor, A, B, out, bwd: bool) -> int:
    """Shapes of a linear call; returns the adapter rank r. The library sees only pointers and
    M, so a tensor of the wrong shape would be read or written out of bounds: it is refused
    here. Forward: x (M, k_in) -> h (M, n_out); input gradient: grad_h (M, n_out) ->
    grad_x (M, k_in); A (r, k_in) and B (n_out, r) together, or neither."""
    name = "grad_h" if bwd else "x"
    if act.dim() != 2:
        raise ValueError(f"{name} must be 2-D (tokens x features)")
    M = act.shape[0]
    _expect_shape(act, (M, n_out if bwd else k_in), name)
    if (A is None) != (B is None):
        raise ValueError("A and B are given together or not at all")
    r = 0
    if A is not None:
        if A.dim() != 2:
            raise ValueError("A must be 2-D (r x k_in)")
        r = A.shape[0]
        _expect_shape(A, (r, k_in), "A")
        _expect_shape(B, (n_out, r), "B")
    if out is not None:
        _expect_shape(out, (M, k_in if bwd else n_out), "out")
    return r


def new_workspace(need: int, device="cuda") -> torch.Tensor:
    """A linear-layer workspace of `need` bytes, all zero as the header asks of a new workspace (see
    qlora_workspace_size there); reusable across calls in stream order."""
    return torch.zeros(max(need, 256), dtype=torch.uint8, device=device)


def workspace_check(ws: torch.Tensor, stream=None):
    """Raise QNError(QN_ETIMEOUT) if a kernel that used `ws` gave up a bounded wait since the last
    check (the error word is then cleared); synchronises the stream."""
    _check(load().qlora_workspace_check(_ptr(ws), _stream(stream)), "qlora_workspace_check")


def selftest_wait_timeout(ws: torch.Tensor, stream=None):
    """Enqueue the library's bounded-wait self-test on a zeroed workspace: its wait runs out and
    sets the error word (see qn_selftest_wait_timeout in the header)."""
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _check(load().qn_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "qn_selftest_wait_timeout")


def _workspace(ws: torch.Tensor | None, need: int, device) -> tuple[torch.Tensor, int]:
    """A caller workspace (contiguous CUDA memory, any dtype) or a fresh one; its size in bytes."""
    if ws is None:
        ws = new_workspace(need, device)
    elif not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ws, ws.numel() * ws.element_size()


def _same_device(w, *ts):
    dev = w.codes.device
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"tensor on {t.device}, the weight is on {dev}")


def sizes(n_out: int, k_in: int):
    """(codes, absmax_q, group_scale, absmax_mean) byte sizes of a quantised weight."""
    a, b, c, d = (ctypes.c_size_t() for _ in range(4))
    _check(load().qn_nf4_sizes(n_out, k_in, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c), ctypes.byref(d)),
           "qn_nf4_sizes")
    return a.value, b.value, c.value, d.value


def weight_sizes(n_out: int, k_in: int, double_quant: bool = True):
    """(codes, absmax_q, group_scale, absmax_mean, absmax fp32) byte sizes for a constant format."""
    v = [ctypes.c_size_t() for _ in range(5)]
    _check(load().qn_weight_sizes(n_out, k_in, CONST_DQ if double_quant else CONST_F32, *(ctypes.byref(x) for x in v)),
           "qn_weight_sizes")
    return tuple(x.value for x in v)


def quantize_workspace_size(n_out: int, k_in: int) -> int:
    v = ctypes.c_size_t()
    _check(load().qn_quantize_workspace_size(n_out, k_in, ctypes.byref(v)), "qn_quantize_workspace_size")
    return v.value


def linear_workspace_size(M: int, n_out: int, k_in: int, r: int) -> int:
    v = ctypes.c_size_t()
    _check(load().qlora_workspace_size(M, n_out, k_in, r, ctypes.byref(v)), "qlora_workspace_size")
    return v.value


def launch_count(reset: bool = False) -> int:
    return int(load().qn_launch_count(1 if reset else 0))


@dataclasses.dataclass
class NF4Weight:
    """A quantised weight: its device buffers plus the shape and format (see include/qlora_nf4.h).
    quant_type "nf4" or "fp4"; double_quant True: absmax_q, group_scale, absmax_mean hold the
    constants; False: absmax (fp32 per block) does, and the other three are empty."""
    n_out: int
    k_in: int
    codes: torch.Tensor        # uint8 [n_out*k_in/2]
    absmax_q: torch.Tensor     # uint8 [nb], E4M3 bits
    group_scale: torch.Tensor  # float32 [ng]
    absmax_mean: torch.Tensor  # float32 [1]
    quant_type: str = "nf4"
    double_quant: bool = True
    absmax: torch.Tensor | None = None  # float32 [nb] (double_quant False)

    @staticmethod
    def empty(n_out: int, k_in: int, device="cuda", quant_type: str = "nf4", double_quant: bool = True) -> "NF4Weight":
        if quant_type not in QUANT_TYPES:
            raise ValueError(f"quant_type {quant_type!r} is not one of {sorted(QUANT_TYPES)}")
        cb, ab, sb, mb, fb = weight_sizes(n_out, k_in, double_quant)
        u8 = dict(dtype=torch.uint8, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        return NF4Weight(n_out, k_in, torch.empty(cb, **u8), torch.empty(ab, **u8), torch.empty(sb // 4, **f32),
                         torch.empty(mb // 4, **f32), quant_type, bool(double_quant),
                         None if double_quant else torch.empty(fb // 4, **f32))

    def c_struct(self) -> CWeight:
        if self.double_quant:
            return CWeight(self.n_out, self.k_in, self.codes.data_ptr(), self.absmax_q.data_ptr(),
                           self.group_scale.data_ptr(), self.absmax_mean.data_ptr(), QUANT_TYPES[self.quant_type],
                           CONST_DQ, None)
        return CWeight(self.n_out, self.k_in, self.codes.data_ptr(), None, None, None, QUANT_TYPES[self.quant_type],
                       CONST_F32, self.absmax.data_ptr())

    def nbytes(self) -> int:
        ts = (self.codes, self.absmax_q, self.group_scale, self.absmax_mean) + (
            () if self.absmax is None else (self.absmax,))
        return sum(t.numel() * t.element_size() for t in ts)


def nf4_quantize(W: torch.Tensor, out: NF4Weight | None = None, workspace: torch.Tensor | None = None,
                 stream=None, quant_type: str = "nf4", double_quant: bool = True) -> NF4Weight:
    """Quantise a bf16 (n_out x k_in) CUDA tensor: NF4 (or "fp4") codes with double-quantised (or
    fp32) block constants; an `out` given keeps its own format."""
    _dev_bf16(W, "W")
    if W.dim() != 2:
        raise ValueError("W must be 2-D (n_out x k_in)")
    n, k = W.shape
    out = out or NF4Weight.empty(n, k, W.device, quant_type, double_quant)
    if (out.n_out, out.k_in) != (n, k):
        raise ValueError(f"out holds a {out.n_out} x {out.k_in} weight, W is {n} x {k}")
    _same_device(out, W)
    workspace, ws_bytes = _workspace(workspace, quantize_workspace_size(n, k), W.device)
    cw = out.c_struct()
    _check(load().nf4_quantize(_ptr(W), ctypes.byref(cw), _ptr(workspace), ws_bytes, _stream(stream)),
           "nf4_quantize")
    return out


def nf4_quantize_static_ws(W: torch.Tensor, out: NF4Weight, stream=None) -> NF4Weight:
    """nf4_quantize using the library's static device scratch instead of a workspace; the
    library allocates nothing (the output buffers are the caller's). See the header for the
    size limit and the rule that overlapping calls race."""
    _dev_bf16(W, "W")
    if W.dim() != 2 or (out.n_out, out.k_in) != tuple(W.shape):
        raise ValueError(f"W of shape {tuple(W.shape)} does not match a {out.n_out} x {out.k_in} weight")
    _same_device(out, W)
    cw = out.c_struct()
    _check(load().nf4_quantize_static_ws(_ptr(W), ctypes.byref(cw), _stream(stream)), "nf4_quantize_static_ws")
    return out


def nf4_dequantize(w: NF4Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    out = out if out is not None else torch.empty(w.n_out, w.k_in, dtype=torch.bfloat16, device=w.codes.device)
    _dev_bf16(out, "out")
    _expect_shape(out, (w.n_out, w.k_in), "out")
    _same_device(w, out)
    cw = w.c_struct()
    _check(load().nf4_dequantize(ctypes.byref(cw), _ptr(out), _stream(stream)), "nf4_dequantize")
    return out


def _lora(A, B, r):
    if r == 0:
        return None, None
    _dev_bf16(A, "A")
    _dev_bf16(B, "B")
    return A, B


def qlora_linear_fwd(w: NF4Weight, x: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None,
                     alpha: float, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None, dropout=None) -> torch.Tensor:
    """h = dequant(W) x + (alpha/r) B (A x); x is M x k_in, h is M x n_out (bf16).
    dropout = (p, seed, offset): LoRA dropout of the adapter's input (qlora_linear_fwd_dropout)."""
    _dev_bf16(x, "x")
    r = check_linear_shapes(w.n_out, w.k_in, x, A, B, out, bwd=False)
    M = x.shape[0]
    A, B = _lora(A, B, r)
    out = out if out is not None else torch.empty(M, w.n_out, dtype=torch.bfloat16, device=x.device)
    _dev_bf16(out, "out")
    _same_device(w, x, A, B, out)
    workspace, ws_bytes = _workspace(workspace, linear_workspace_size(M, w.n_out, w.k_in, r), x.device)
    cw = w.c_struct()
    if dropout is None:
        _check(load().qlora_linear_fwd(ctypes.byref(cw), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(out),
                                       _ptr(workspace), ws_bytes, _stream(stream)), "qlora_linear_fwd")
    else:
        d = _dropout_struct(dropout)
        _check(load().qlora_linear_fwd_dropout(ctypes.byref(cw), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha),
                                               ctypes.byref(d), _ptr(out), _ptr(workspace), ws_bytes,
                                               _stream(stream)), "qlora_linear_fwd_dropout")
    return out


def qlora_linear_bwd_x(w: NF4Weight, grad_h: torch.Tensor, A: torch.Tensor | None, B: torch.Tensor | None,
                       alpha: float, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None, dropout=None) -> torch.Tensor:
    """grad_x = dequant(W)^T grad_h + (alpha/r) A^T (B^T grad_h); grad_h is M x n_out.
    dropout = (p, seed, offset): the forward's LoRA-dropout mask (qlora_linear_bwd_x_dropout)."""
    _dev_bf16(grad_h, "grad_h")
    r = check_linear_shapes(w.n_out, w.k_in, grad_h, A, B, out, bwd=True)
    M = grad_h.shape[0]
    A, B = _lora(A, B, r)
    out = out if out is not None else torch.empty(M, w.k_in, dtype=torch.bfloat16, device=grad_h.device)
    _dev_bf16(out, "out")
    _same_device(w, grad_h, A, B, out)
    workspace, ws_bytes = _workspace(workspace, linear_workspace_size(M, w.n_out, w.k_in, r), grad_h.device)
    cw = w.c_struct()
    if dropout is None:
        _check(load().qlora_linear_bwd_x(ctypes.byref(cw), _ptr(grad_h), M, _ptr(A), _ptr(B), r, float(alpha),
                                         _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
               "qlora_linear_bwd_x")
    else:
        d = _dropout_struct(dropout)
        _check(load().qlora_linear_bwd_x_dropout(ctypes.byref(cw), _ptr(grad_h), M, _ptr(A), _ptr(B), r,
                                                 float(alpha), ctypes.byref(d), _ptr(out), _ptr(workspace),
                                                 ws_bytes, _stream(stream)), "qlora_linear_bwd_x_dropout")
    return out


def qlora_merge_bf16(w: NF4Weight, A: torch.Tensor | None, B: torch.Tensor | None, alpha: float,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W' + (alpha/r) B A as a bf16 n_out x k_in tensor (merge and unload)."""
    if (A is None) != (B is None):
        raise ValueError("A and B are given together or not at all")
    r = 0
    if A is not None:
        _dev_bf16(A, "A")
        _dev_bf16(B, "B")
        if A.dim() != 2:
            raise ValueError("A must be 2-D (r x k_in)")
        r = A.shape[0]
        _expect_shape(A, (r, w.k_in), "A")
        _expect_shape(B, (w.n_out, r), "B")
    out = out if out is not None else torch.empty(w.n_out, w.k_in, dtype=torch.bfloat16, device=w.codes.device)
    _dev_bf16(out, "out")
    _expect_shape(out, (w.n_out, w.k_in), "out")
    _same_device(w, A, B, out)
    cw = w.c_struct()
    _check(load().qlora_merge_bf16(ctypes.byref(cw), _ptr(A), _ptr(B), r, float(alpha), _ptr(out), _stream(stream)),
           "qlora_merge_bf16")
    return out


def lora_grads_workspace_size(M: int, r: int) -> int:
    v = ctypes.c_size_t()
    _check(load().qlora_lora_grads_workspace_size(M, r, ctypes.byref(v)), "qlora_lora_grads_workspace_size")
    return v.value


def qlora_lora_grads(x: torch.Tensor, grad_h: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                     grad_A: torch.Tensor | None = None, grad_B: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None, dropout=None):
    """(grad_A (r x k_in), grad_B (n_out x r)) in fp32 for x (M x k_in) and grad_h (M x n_out).
    dropout = (p, seed, offset): the forward's LoRA-dropout mask (qlora_lora_grads_dropout)."""
    for t, nm in ((x, "x"), (grad_h, "grad_h"), (A, "A"), (B, "B")):
        _dev_bf16(t, nm)
    if x.dim() != 2 or grad_h.dim() != 2 or A.dim() != 2 or B.dim() != 2:
        raise ValueError("x, grad_h, A and B must be 2-D")
    M, k = x.shape
    n = grad_h.shape[1]
    r = A.shape[0]
    _expect_shape(grad_h, (M, n), "grad_h")
    _expect_shape(A, (r, k), "A")
    _expect_shape(B, (n, r), "B")
    f32 = dict(dtype=torch.float32, device=x.device)
    grad_A = grad_A if grad_A is not None else torch.empty(r, k, **f32)
    grad_B = grad_B if grad_B is not None else torch.empty(n, r, **f32)
    for t, shp, nm in ((grad_A, (r, k), "grad_A"), (grad_B, (n, r), "grad_B")):
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous fp32 CUDA tensor")
        _expect_shape(t, shp, nm)
    if workspace is None:
        workspace = torch.empty(max(lora_grads_workspace_size(M, r), 256), dtype=torch.uint8, device=x.device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    for t in (grad_h, A, B, grad_A, grad_B, workspace):
        if t.device != x.device:
            raise ValueError(f"tensor on {t.device}, x is on {x.device}")
    wsb = workspace.numel() * workspace.element_size()
    if dropout is None:
        _check(load().qlora_lora_grads(_ptr(x), _ptr(grad_h), M, n, k, _ptr(A), _ptr(B), r, float(alpha),
                                       _ptr(grad_A), _ptr(grad_B), _ptr(workspace), wsb, _stream(stream)),
               "qlora_lora_grads")
    else:
        d = _dropout_struct(dropout)
        _check(load().qlora_lora_grads_dropout(_ptr(x), _ptr(grad_h), M, n, k, _ptr(A), _ptr(B), r, float(alpha),
                                               ctypes.byref(d), _ptr(grad_A), _ptr(grad_B), _ptr(workspace), wsb,
                                               _stream(stream)), "qlora_lora_grads_dropout")
    return grad_A, grad_B


# ------------------------------------------------------- activations kept in 8 bits
# The calls below run on the tensors' device, which has to be the current one, on the current (or the
# given) stream of it. What they allocate belongs to that stream.

_marshal = None


class _NoMarshal:
    """In place of the compiled marshalling: every call takes the general way."""

    def __getattr__(self, name):
        return lambda *operands: None


def _native():
    """The compiled marshalling of the plain calls (csrc/marshal.cpp): new results, current stream. A call of it gives the
    results, a status, or None when the operands need the general way below, which does the same through the same library
    and takes the host a few microseconds more."""
    global _marshal
    if _marshal is None:
        lib = load()
        from .build import marshal_path
        path = marshal_path()
        if not os.path.exists(path):
            warnings.warn(f"{path} is missing, calls take longer on the host: build it with "
                          "`python -m bit_nf4_quantized_25_b200.build`", RuntimeWarning, stacklevel=3)
            _marshal = _NoMarshal()
            return _marshal
        spec = importlib.util.spec_from_file_location(__package__ + "._marshal", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.act8_quantize, lib.act8_dequantize, lib.qlora_lora_grads_act8_workspace_size, lib.qlora_lora_grads_act8,
            lib.swiglu_act8_fwd, lib.swiglu_act8_bwd, lib.int4_quantize, lib.int4_dequantize, lib.int4_linear_fwd)))
        _marshal = m
    return _marshal


def _stream_here(dev: torch.device, stream=None) -> int:
    """The stream's handle, after checking that `dev` is the device that the library would launch on."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors are on {dev}, not on a CUDA device")
    here = torch._C._cuda_getDevice()
    if dev.index != here:
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{here}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(here)
    if stream.device_index != here:
        raise ValueError(f"the stream is one of cuda:{stream.device_index}, the current device is cuda:{here}")
    return stream.cuda_stream


def _expect(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: torch.device, part: str = ""):
    """t is a contiguous tensor of this type and shape on `dev`: the library sees only its address."""
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}{part} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _done(r, what: str):
    """What a native call gave, unless it is a status."""
    if type(r) is int:
        _check(r, what)
    return r


def _new(stream, make, *args, **kw):
    """make(...) in the allocations of the stream that the call runs on: memory that another stream has freed may
    still be in use there, and a workspace dropped at return must not go to another stream before the kernels end."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2 or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a 2-D bf16 tensor, got {t.dtype} of shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.shape


@functools.lru_cache(maxsize=1024)  # asked for with every new buffer
def act8_sizes(rows: int, cols: int):
    """(codes, absmax) byte sizes of an activation in 8 bits."""
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().qn_act8_sizes(rows, cols, ctypes.byref(a), ctypes.byref(b)), "qn_act8_sizes")
    return a.value, b.value


@dataclasses.dataclass
class Act8:
    """An activation in 8 bits (see qn_act8 in include/qlora_nf4.h): a row's 64 consecutive values share an
    absmax; a value is codes * absmax / 127."""
    rows: int
    cols: int
    codes: torch.Tensor   # int8 [rows, cols]
    absmax: torch.Tensor  # bfloat16 [rows, cols / 64]

    @staticmethod
    def empty(rows: int, cols: int, device="cuda") -> "Act8":
        act8_sizes(rows, cols)  # refuses what the format does not hold
        return Act8(rows, cols, torch.empty(rows, cols, dtype=torch.int8, device=device),
                    torch.empty(rows, cols // BLOCK, dtype=torch.bfloat16, device=device))

    def c_struct(self, dev: torch.device, name: str = "Act8") -> CAct8:
        _expect(self.codes, name, torch.int8, (self.rows, self.cols), dev, ".codes")
        _expect(self.absmax, name, torch.bfloat16, (self.rows, self.cols // BLOCK), dev, ".absmax")
        return self._c()

    def _c(self) -> CAct8:  # of checked buffers, or new ones
        return CAct8(self.rows, self.cols, self.codes.data_ptr(), self.absmax.data_ptr())

    def nbytes(self) -> int:
        return self.codes.numel() + 2 * self.absmax.numel()


def act8_quantize(x: torch.Tensor, out: Act8 | None = None, stream=None) -> Act8:
    """An activation (M x k, bf16) in 8 bits, to keep for the backward pass."""
    if out is None and stream is None:
        r = _native().act8_quantize(x)
        if r is not None:
            return Act8(*x.shape, *_done(r, "act8_quantize"))
    M, k = _matrix(x, "x")
    s = _stream_here(x.device, stream)
    if out is None:
        out = _new(stream, Act8.empty, M, k, x.device)
        c = out._c()
    elif (out.rows, out.cols) != (M, k):
        raise ValueError(f"out holds {out.rows} x {out.cols} values, x is {M} x {k}")
    else:
        c = out.c_struct(x.device, "out")
    st = load().act8_quantize(x.data_ptr(), ctypes.byref(c), s)
    if st != QN_OK:
        _check(st, "act8_quantize")
    return out


def act8_dequantize(a: Act8, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The bf16 values of an activation in 8 bits."""
    if out is None and stream is None:
        r = _native().act8_dequantize(a.rows, a.cols, a.codes, a.absmax)
        if r is not None:
            return _done(r, "act8_dequantize")
    dev = a.codes.device
    s = _stream_here(dev, stream)
    if out is None:
        out = _new(stream, torch.empty, a.rows, a.cols, dtype=torch.bfloat16, device=dev)
    else:
        _expect(out, "out", torch.bfloat16, (a.rows, a.cols), dev)
    st = load().act8_dequantize(ctypes.byref(a.c_struct(dev, "a")), out.data_ptr(), s)
    if st != QN_OK:
        _check(st, "act8_dequantize")
    return out


@functools.lru_cache(maxsize=1024)
def lora_grads_act8_workspace_size(M: int, n_out: int, r: int) -> int:
    v = ctypes.c_size_t()
    _check(load().qlora_lora_grads_act8_workspace_size(M, n_out, r, ctypes.byref(v)),
           "qlora_lora_grads_act8_workspace_size")
    return v.value


def qlora_lora_grads_act8(x: Act8, grad_h: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                          grad_A: torch.Tensor | None = None, grad_B: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None, dropout=None):
    """(grad_A (r x k_in), grad_B (n_out x r)) in fp32 for an input x kept in 8 bits and grad_h (M x n_out).
    dropout = (p, seed, offset): the forward's LoRA-dropout mask."""
    if grad_A is None and grad_B is None and workspace is None and stream is None and dropout is None:
        r = _native().lora_grads(x.rows, x.cols, x.codes, x.absmax, grad_h, A, B, float(alpha))
        if r is not None:
            return _done(r, "qlora_lora_grads_act8")
    return _grads_act8(load().qlora_lora_grads_act8, "qlora_lora_grads_act8", x, grad_h, A, B, alpha, grad_A, grad_B,
                       workspace, stream, dropout)


def selftest_grads_give_up(x: Act8, grad_h: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float, dropout,
                           stream=None):
    """qlora_lora_grads_act8 in which waits run out (see qn_selftest_grads_give_up in the header): grad_A is NaN."""
    return _grads_act8(load().qn_selftest_grads_give_up, "qn_selftest_grads_give_up", x, grad_h, A, B, alpha, None, None,
                       None, stream, dropout)


def _grads_act8(call, what: str, x, grad_h, A, B, alpha, grad_A, grad_B, workspace, stream, dropout):
    M, k = x.rows, x.cols
    n = _matrix(grad_h, "grad_h")[1]
    r = _matrix(A, "A")[0]
    dev = grad_h.device
    s = _stream_here(dev, stream)
    bf, f32 = torch.bfloat16, torch.float32
    _expect(grad_h, "grad_h", bf, (M, n), dev)
    _expect(A, "A", bf, (r, k), dev)
    _expect(B, "B", bf, (n, r), dev)
    cx = x.c_struct(dev, "x")
    if grad_A is None:
        grad_A = _new(stream, torch.empty, r, k, dtype=f32, device=dev)
    else:
        _expect(grad_A, "grad_A", f32, (r, k), dev)
    if grad_B is None:
        grad_B = _new(stream, torch.empty, n, r, dtype=f32, device=dev)
    else:
        _expect(grad_B, "grad_B", f32, (n, r), dev)
    if workspace is None:
        workspace = _new(stream, torch.empty, lora_grads_act8_workspace_size(M, n, r), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    d = None if dropout is None else ctypes.byref(_dropout_struct(dropout))
    _check(call(ctypes.byref(cx), grad_h.data_ptr(), n, A.data_ptr(), B.data_ptr(), r, float(alpha), d, grad_A.data_ptr(),
                grad_B.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), s), what)
    return grad_A, grad_B


def swiglu_act8_fwd(gate: torch.Tensor, up: torch.Tensor, out: torch.Tensor | None = None, gate8: Act8 | None = None,
                    up8: Act8 | None = None, stream=None):
    """(y, gate8, up8): y = silu(gate) * up in bf16, and gate and up in 8 bits for swiglu_act8_bwd."""
    if out is None and gate8 is None and up8 is None and stream is None:
        r = _native().swiglu_fwd(gate, up)
        if r is not None:
            y, gc, ga, uc, ua = _done(r, "swiglu_act8_fwd")
            M, n = gate.shape
            return y, Act8(M, n, gc, ga), Act8(M, n, uc, ua)
    M, n = _matrix(gate, "gate")
    dev = gate.device
    s = _stream_here(dev, stream)
    _expect(up, "up", torch.bfloat16, (M, n), dev)
    kept, structs = [], []
    for a, nm in ((gate8, "gate8"), (up8, "up8")):
        if a is None:
            a = _new(stream, Act8.empty, M, n, dev)
            structs.append(a._c())
        elif (a.rows, a.cols) != (M, n):
            raise ValueError(f"{nm} holds {a.rows} x {a.cols} values, gate is {M} x {n}")
        else:
            structs.append(a.c_struct(dev, nm))
        kept.append(a)
    if out is None:
        out = _new(stream, torch.empty_like, gate)
    else:
        _expect(out, "out", torch.bfloat16, (M, n), dev)
    st = load().swiglu_act8_fwd(gate.data_ptr(), up.data_ptr(), out.data_ptr(), ctypes.byref(structs[0]),
                                ctypes.byref(structs[1]), s)
    if st != QN_OK:
        _check(st, "swiglu_act8_fwd")
    return out, kept[0], kept[1]


def swiglu_act8_bwd(gate8: Act8, up8: Act8, grad_y: torch.Tensor, grad_gate: torch.Tensor | None = None,
                    grad_up: torch.Tensor | None = None, y8: Act8 | None = None, stream=None, recompute: bool = True):
    """(grad_gate, grad_up, y8) from what swiglu_act8_fwd kept; y8 is y once more, in 8 bits, the input that the
    next layer's adapter gradients take (None with recompute=False)."""
    M, n = gate8.rows, gate8.cols
    if grad_gate is None and grad_up is None and y8 is None and stream is None and recompute:
        r = _native().swiglu_bwd(M, n, gate8.codes, gate8.absmax, up8.rows, up8.cols, up8.codes, up8.absmax, grad_y)
        if r is not None:
            gg, gu, yc, ya = _done(r, "swiglu_act8_bwd")
            return gg, gu, Act8(M, n, yc, ya)
    dev = gate8.codes.device
    s = _stream_here(dev, stream)
    _expect(grad_y, "grad_y", torch.bfloat16, (M, n), dev)
    if (up8.rows, up8.cols) != (M, n):
        raise ValueError(f"up8 holds {up8.rows} x {up8.cols} values, gate8 {M} x {n}")
    cy = None
    if y8 is None:
        if recompute:
            y8 = _new(stream, Act8.empty, M, n, dev)
            cy = ctypes.byref(y8._c())
    elif not recompute:
        raise ValueError("y8 is given with recompute=False")
    elif (y8.rows, y8.cols) != (M, n):
        raise ValueError(f"y8 holds {y8.rows} x {y8.cols} values, gate8 {M} x {n}")
    else:
        cy = ctypes.byref(y8.c_struct(dev, "y8"))
    grads = []
    for t, nm in ((grad_gate, "grad_gate"), (grad_up, "grad_up")):
        if t is None:
            t = _new(stream, torch.empty_like, grad_y)
        else:
            _expect(t, nm, torch.bfloat16, (M, n), dev)
        grads.append(t)
    st = load().swiglu_act8_bwd(ctypes.byref(gate8.c_struct(dev, "gate8")), ctypes.byref(up8.c_struct(dev, "up8")),
                                grad_y.data_ptr(), grads[0].data_ptr(), grads[1].data_ptr(), cy, s)
    if st != QN_OK:
        _check(st, "swiglu_act8_bwd")
    return grads[0], grads[1], y8


# ------------------------------------------- 4-bit integer weights with group scales

@functools.lru_cache(maxsize=1024)
def int4_sizes(n_out: int, k_in: int, group: int):
    """(codes, scale, zero_point) byte sizes of a weight in 4-bit integers."""
    v = [ctypes.c_size_t() for _ in range(3)]
    _check(load().qn_int4_sizes(n_out, k_in, group, *(ctypes.byref(x) for x in v)), "qn_int4_sizes")
    return tuple(x.value for x in v)


@dataclasses.dataclass
class Int4Weight:
    """A weight in 4-bit integers (see qn_int4_weight in include/qlora_nf4.h): scale * (code - zero_point), with a
    scale and a zero point for each `group` consecutive weights of a row; without zero_point it is 8."""
    n_out: int
    k_in: int
    group: int
    codes: torch.Tensor                     # uint8 [n_out, k_in / 2]
    scale: torch.Tensor                     # bfloat16 [n_out, k_in / group]
    zero_point: torch.Tensor | None = None  # uint8 [n_out, k_in / group], 0..15

    @staticmethod
    def empty(n_out: int, k_in: int, group: int = 128, zero_point: bool = True, device="cuda") -> "Int4Weight":
        int4_sizes(n_out, k_in, group)  # refuses what the format does not hold
        return Int4Weight(n_out, k_in, group, torch.empty(n_out, k_in // 2, dtype=torch.uint8, device=device),
                          torch.empty(n_out, k_in // group, dtype=torch.bfloat16, device=device),
                          torch.empty(n_out, k_in // group, dtype=torch.uint8, device=device) if zero_point else None)

    def c_struct(self, dev: torch.device) -> CInt4:
        if self.group not in (32, 64, 128):
            raise ValueError(f"group {self.group} is not 32, 64 or 128")
        groups = (self.n_out, self.k_in // self.group)
        _expect(self.codes, "codes", torch.uint8, (self.n_out, self.k_in // 2), dev)
        _expect(self.scale, "scale", torch.bfloat16, groups, dev)
        if self.zero_point is not None:
            _expect(self.zero_point, "zero_point", torch.uint8, groups, dev)
        return self._c()

    def _c(self) -> CInt4:  # of checked buffers, or new ones
        z = self.zero_point
        return CInt4(self.n_out, self.k_in, self.group, self.codes.data_ptr(), self.scale.data_ptr(),
                     None if z is None else z.data_ptr())

    def nbytes(self) -> int:
        return self.codes.numel() + 2 * self.scale.numel() + (0 if self.zero_point is None else self.zero_point.numel())


def int4_quantize(W: torch.Tensor, out: Int4Weight | None = None, group: int = 128, zero_point: bool = True,
                  stream=None) -> Int4Weight:
    """Quantise a bf16 (n_out x k_in) weight, a merged one for instance, to 4-bit integers; an `out` given keeps its
    own group and zero points."""
    if out is None and stream is None:
        r = _native().int4_quantize(W, group, zero_point)
        if r is not None:
            return Int4Weight(*W.shape, group, *_done(r, "int4_quantize"))
    n, k = _matrix(W, "W")
    s = _stream_here(W.device, stream)
    if out is None:
        out = _new(stream, Int4Weight.empty, n, k, group, zero_point, W.device)
        c = out._c()
    elif (out.n_out, out.k_in) != (n, k):
        raise ValueError(f"out holds a {out.n_out} x {out.k_in} weight, W is {n} x {k}")
    else:
        c = out.c_struct(W.device)
    st = load().int4_quantize(W.data_ptr(), ctypes.byref(c), s)
    if st != QN_OK:
        _check(st, "int4_quantize")
    return out


def int4_dequantize(w: Int4Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The bf16 weight that w stands for."""
    if out is None and stream is None:
        r = _native().int4_dequantize(w.n_out, w.k_in, w.group, w.codes, w.scale, w.zero_point)
        if r is not None:
            return _done(r, "int4_dequantize")
    dev = w.codes.device
    s = _stream_here(dev, stream)
    if out is None:
        out = _new(stream, torch.empty, w.n_out, w.k_in, dtype=torch.bfloat16, device=dev)
    else:
        _expect(out, "out", torch.bfloat16, (w.n_out, w.k_in), dev)
    _check(load().int4_dequantize(ctypes.byref(w.c_struct(dev)), out.data_ptr(), s), "int4_dequantize")
    return out


def int4_linear_fwd(w: Int4Weight, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h = dequant(W) x for at most 64 tokens; x is M x k_in, h is M x n_out (bf16)."""
    if out is None and stream is None:
        r = _native().int4_linear(w.n_out, w.k_in, w.group, w.codes, w.scale, w.zero_point, x)
        if r is not None:
            return _done(r, "int4_linear_fwd")
    dev = x.device
    s = _stream_here(dev, stream)
    M = _matrix(x, "x")[0]
    if x.shape[1] != w.k_in:
        raise ValueError(f"x has shape {tuple(x.shape)}, the weight takes {w.k_in} features")
    if out is None:
        out = _new(stream, torch.empty, M, w.n_out, dtype=torch.bfloat16, device=dev)
    else:
        _expect(out, "out", torch.bfloat16, (M, w.n_out), dev)
    st = load().int4_linear_fwd(ctypes.byref(w.c_struct(dev)), x.data_ptr(), M, out.data_ptr(), s)
    if st != QN_OK:
        _check(st, "int4_linear_fwd")
    return out
