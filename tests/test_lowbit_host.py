"""Host-side checks of the 8-bit activation and 4-bit integer entry points: sizes, refusals before anything
is enqueued (the addresses here are never read: no call reaches a GPU), and the binding's own checks."""
import ctypes

import pytest
import torch

import lowbit_ref as ref


@pytest.fixture(scope="module")
def qb():
    from bit_nf4_quantized_25_b200 import binding, build
    build.build()
    binding.load()
    return binding


@pytest.fixture(scope="module")
def lib(qb):
    return qb.load()


P = ctypes.c_void_p
OK, EINVAL, ESHAPE, EALIGN = 0, 1, 2, 3


def _act8(qb, rows=4, cols=128, base=0x100000, absmax=None):
    return qb.CAct8(rows, cols, base, base + 0x10000 if absmax is None else absmax)


def _int4(qb, n=32, k=256, group=64, base=0x100000, zero=True):
    return qb.CInt4(n, k, group, base, base + 0x10000, base + 0x20000 if zero else None)


def test_act8_sizes(lib, qb):
    assert qb.act8_sizes(3, 192) == (576, 18)
    assert qb.act8_sizes(0, 64) == (0, 0)
    big = qb.act8_sizes(1 << 20, 28672)  # beyond 32 bits
    assert big == ((1 << 20) * 28672, (1 << 20) * 28672 // 32)
    assert 8 * sum(qb.act8_sizes(4096, 4096)) / 4096 ** 2 == 8.25
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    for rows, cols, want in ((4, 96, ESHAPE), (-1, 64, EINVAL), (4, -64, EINVAL), (1 << 31, 64, ESHAPE),
                             ((1 << 31) - 1, 1 << 30, ESHAPE)):
        assert lib.qn_act8_sizes(rows, cols, ctypes.byref(a), ctypes.byref(b)) == want, (rows, cols)
    assert lib.qn_act8_sizes(4, 64, None, ctypes.byref(b)) == EINVAL


def test_act8_refusals(lib, qb):
    f, r = lib.act8_quantize, ctypes.byref
    x = P(0x400000)
    assert f(x, None, None) == EINVAL
    assert f(None, r(_act8(qb)), None) == EINVAL
    assert f(P(0x400008), r(_act8(qb)), None) == EALIGN
    assert f(x, r(_act8(qb, cols=100)), None) == ESHAPE
    assert f(x, r(_act8(qb, base=0x100004)), None) == EALIGN
    assert f(x, r(_act8(qb, absmax=0x300001)), None) == EALIGN
    assert f(x, r(qb.CAct8(4, 128, None, 0x300000)), None) == EINVAL
    assert f(x, r(qb.CAct8(4, 128, 0x300000, None)), None) == EINVAL
    assert f(P(0x100000), r(_act8(qb)), None) == EINVAL  # codes over x
    assert f(x, r(_act8(qb, absmax=0x400010)), None) == EINVAL  # absmax inside x
    assert "overlaps" in lib.qn_last_error().decode()
    g = lib.act8_dequantize
    assert g(None, x, None) == EINVAL
    assert g(r(_act8(qb)), None, None) == EINVAL
    assert g(r(_act8(qb)), P(0x400002), None) == EALIGN
    assert g(r(_act8(qb)), P(0x100000 - 512), None) == EINVAL  # the last bytes of the output are codes
    before = lib.qn_launch_count(0)
    assert f(None, r(_act8(qb, rows=0)), None) == OK and g(r(_act8(qb, cols=0)), None, None) == OK
    assert lib.qn_launch_count(0) == before


def test_swiglu_refusals(lib, qb):
    r = ctypes.byref
    g8, u8, y8 = _act8(qb), _act8(qb, base=0x200000), _act8(qb, base=0x300000)
    g, u, y, d = P(0x400000), P(0x500000), P(0x600000), P(0x700000)
    f = lib.swiglu_act8_fwd
    assert f(None, u, y, r(g8), r(u8), None) == EINVAL
    assert f(g, u, P(0x600004), r(g8), r(u8), None) == EALIGN
    assert f(g, u, y, r(g8), r(_act8(qb, rows=5, base=0x200000)), None) == ESHAPE
    assert f(g, u, y, r(g8), None, None) == EINVAL
    assert f(g, u, g, r(g8), r(u8), None) == EINVAL  # in place
    assert f(g, u, y, r(g8), r(g8), None) == EINVAL  # one buffer for both
    b = lib.swiglu_act8_bwd
    assert b(r(g8), r(u8), None, y, d, None, None) == EINVAL
    assert b(r(g8), r(u8), g, y, y, None, None) == EINVAL  # both gradients in one buffer
    assert b(r(g8), r(u8), g, g, d, None, None) == EINVAL  # over grad_y
    assert b(r(g8), r(u8), g, y, d, r(g8), None) == EINVAL  # y8 over gate8
    assert b(r(g8), r(u8), g, y, d, r(_act8(qb, cols=64, base=0x300000)), None) == ESHAPE
    assert b(r(g8), r(u8), P(0x400001), y, d, r(y8), None) == EALIGN
    before = lib.qn_launch_count(0)
    e = _act8(qb, rows=0)
    assert f(None, None, None, r(e), r(e), None) == OK and b(r(e), r(e), None, None, None, None, None) == OK
    assert lib.qn_launch_count(0) == before


def test_lora_grads_act8_refusals(lib, qb):
    r = ctypes.byref
    x = _act8(qb)  # 4 x 128
    gh, A, B, ga, gb, ws = (P(0x400000 + 0x100000 * i) for i in range(6))
    f = lib.qlora_lora_grads_act8
    size = qb.lora_grads_act8_workspace_size(4, 96, 16)
    assert size >= 2 * 16 * 16 * 4

    def call(x=x, gh=gh, n=96, A=A, B=B, rank=16, alpha=32.0, d=None, ga=ga, gb=gb, ws=ws, size=size):
        return f(None if x is None else r(x), gh, n, A, B, rank, alpha, None if d is None else r(d), ga, gb, ws, size,
                 None)

    assert call(x=None) == EINVAL
    assert call(x=_act8(qb, cols=96)) == ESHAPE
    assert call(x=qb.CAct8(4, 128, None, 0x110000)) == EINVAL
    assert call(n=-1) == EINVAL
    assert call(rank=0) == EINVAL and call(rank=257, size=1 << 20) == EINVAL
    assert call(alpha=float("inf")) == EINVAL and call(alpha=float("nan")) == EINVAL
    assert call(d=qb.CDropout(1.0, 1, 0)) == EINVAL and call(d=qb.CDropout(float("nan"), 1, 0)) == EINVAL
    assert call(gh=None) == EINVAL and call(A=None) == EINVAL and call(B=None) == EINVAL
    assert call(ga=None) == EINVAL and call(gb=None) == EINVAL
    assert call(gh=P(0x400002)) == EALIGN and call(A=P(0x500008)) == EALIGN and call(gb=P(0x800002)) == EALIGN
    assert call(ws=None) == 5 and call(size=size - 1) == 5  # QN_EWORKSPACE
    assert call(ws=P(0x900010)) == EALIGN
    assert call(ga=gb) == EINVAL  # both gradients in one buffer
    assert call(ga=A) == EINVAL and call(gb=P(0x400000 + 64)) == EINVAL and call(ws=ga) == EINVAL
    assert call(ga=P(0x100000)) == EINVAL  # over the codes
    before = lib.qn_launch_count(0)
    assert f(r(qb.CAct8(4, 0, None, None)), None, 0, None, None, 16, 1.0, None, None, None, None, 0, None) == OK
    assert lib.qn_launch_count(0) == before
    v = ctypes.c_size_t()
    assert lib.qlora_lora_grads_act8_workspace_size(-1, 96, 16, r(v)) == EINVAL
    assert lib.qlora_lora_grads_act8_workspace_size(4, -1, 16, r(v)) == EINVAL
    assert lib.qlora_lora_grads_act8_workspace_size(4, 96, 300, r(v)) == EINVAL
    assert lib.qlora_lora_grads_act8_workspace_size(4, 96, 16, None) == EINVAL
    # odd widths of a long batch: a padded copy of grad_h, and of B for odd ranks
    even, odd = (qb.lora_grads_act8_workspace_size(1000, n, 16) for n in (4096, 4097))
    assert odd - even >= 2 * 1000 * 4104
    assert qb.lora_grads_act8_workspace_size(1000, 4096, 13) - even >= 2 * 4096 * 16


def test_int4_sizes(lib, qb):
    assert qb.int4_sizes(32, 256, 64) == (32 * 128, 2 * 32 * 4, 32 * 4)
    assert qb.int4_sizes(5, 64, 32) == (160, 20, 10)
    v = [ctypes.c_size_t() for _ in range(3)]
    out = [ctypes.byref(x) for x in v]
    for n, k, group, want in ((4, 64, 48, EINVAL), (4, 64, 256, EINVAL), (4, 64, 128, ESHAPE), (4, 96, 32, ESHAPE),
                              (-1, 64, 64, EINVAL), ((1 << 31) - 1, 1 << 30, 64, ESHAPE)):
        assert lib.qn_int4_sizes(n, k, group, *out) == want, (n, k, group)
    assert lib.qn_int4_sizes(4, 64, 64, None, *out[1:]) == EINVAL


def test_int4_refusals(lib, qb):
    r = ctypes.byref
    W, x, h = P(0x400000), P(0x500000), P(0x600000)
    for f in (lambda w, m: lib.int4_quantize(m, w, None), lambda w, m: lib.int4_dequantize(w, m, None)):
        assert f(None, W) == EINVAL
        assert f(r(_int4(qb)), None) == EINVAL
        assert f(r(_int4(qb)), P(0x400008)) == EALIGN
        assert f(r(_int4(qb, group=96)), W) == EINVAL
        assert f(r(_int4(qb, k=320, group=128)), W) == ESHAPE
        assert f(r(_int4(qb, base=0x100008)), W) == EALIGN
        assert f(r(qb.CInt4(32, 256, 64, 0x100000, 0x200001, None)), W) == EALIGN
        assert f(r(qb.CInt4(32, 256, 64, 0x100000, None, None)), W) == EINVAL
        assert f(r(_int4(qb)), P(0x110000 - 0x1000)) == EINVAL  # overlap
        assert f(r(_int4(qb, n=0)), None) == OK
    f = lib.int4_linear_fwd
    w = _int4(qb)
    assert f(None, x, 1, h, None) == EINVAL
    assert f(r(w), x, -1, h, None) == EINVAL
    assert f(r(w), x, 65, h, None) == ESHAPE
    assert f(r(_int4(qb, k=65600)), x, 1, h, None) == ESHAPE
    assert f(r(w), None, 1, h, None) == EINVAL
    assert f(r(w), x, 1, None, None) == EINVAL
    assert f(r(w), P(0x500002), 1, h, None) == EALIGN
    assert f(r(w), x, 1, P(0x600008), None) == EALIGN
    assert f(r(w), x, 1, x, None) == EINVAL
    assert f(r(w), x, 1, P(0x110000), None) == EINVAL  # over the scales
    before = lib.qn_launch_count(0)
    assert f(r(w), None, 0, None, None) == OK and f(r(_int4(qb, n=0)), None, 3, None, None) == OK
    assert lib.qn_launch_count(0) == before


def test_the_compiled_marshalling_leaves_what_is_not_plain_to_the_general_way(lib, qb):
    m = qb._native()
    bf = torch.bfloat16
    x, codes, absmax = torch.zeros(2, 64, dtype=bf), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 1, dtype=bf)
    u8 = torch.zeros(2, 32, dtype=torch.uint8)
    for call, operands in ((m.act8_quantize, (x,)), (m.act8_dequantize, (2, 64, codes, absmax)),
                           (m.lora_grads, (2, 64, codes, absmax, x, x, x, 1.0)), (m.swiglu_fwd, (x, x)),
                           (m.swiglu_bwd, (2, 64, codes, absmax, 2, 64, codes, absmax, x)), (m.int4_quantize, (x, 64, True)),
                           (m.int4_dequantize, (2, 64, 64, u8, absmax, None)), (m.int4_linear, (2, 64, 64, u8, absmax, None, x))):
        assert call(*operands) is None  # not on a GPU
        assert call(*(None for _ in operands)) is None
        with pytest.raises(TypeError, match="arguments"):
            call(*operands, 0)
    with pytest.raises(TypeError):
        m.bind(1)
    with pytest.raises(ValueError, match="null"):
        m.bind(*[0] * 9)


def test_binding_refuses_before_the_library(qb):
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="not on a CUDA device"):
        qb.act8_quantize(torch.zeros(2, 64, dtype=bf))
    with pytest.raises(ValueError, match="2-D bf16"):
        qb.act8_quantize(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="contiguous"):
        qb.act8_quantize(torch.zeros(64, 4, dtype=bf).t())
    with pytest.raises(qb.QNError):
        qb.Act8.empty(4, 100, device="cpu")
    with pytest.raises(qb.QNError):
        qb.Int4Weight.empty(4, 192, 128, device="cpu")
    cpu = torch.device("cpu")
    a = qb.Act8.empty(4, 128, device="cpu")
    assert a.c_struct(cpu).rows == 4 and a.nbytes() == 4 * 128 + 2 * 8
    a.absmax = a.absmax.float()
    with pytest.raises(ValueError, match="absmax"):
        a.c_struct(cpu)
    a = qb.Act8(4, 128, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=bf))
    with pytest.raises(ValueError, match="codes"):
        a.c_struct(cpu)
    w = qb.Int4Weight.empty(4, 256, 64, device="cpu")
    assert w.c_struct(cpu).k_in == 256 and w.nbytes() == 4 * 128 + 32 + 16
    for bad in (dict(group=48), dict(scale=w.scale.float()), dict(scale=w.scale[:, :2]), dict(codes=w.codes[:2]),
                dict(zero_point=w.zero_point.int()), dict(zero_point=w.zero_point[:, ::2])):
        import dataclasses
        with pytest.raises(ValueError):
            dataclasses.replace(w, **bad).c_struct(cpu)


# ------------------------------------------------------------- the plain forms themselves

def test_reference_rounds_halves_away_and_marks_blocks():
    x = torch.zeros(1, 192).bfloat16()
    x[0, :4] = torch.tensor([2.0, 1.0, -1.0, -2.0])  # 127 x / a = 127, 63.5, -63.5, -127
    x[0, 130] = float("inf")
    q, a = ref.act8(x)
    assert q[0, :4].tolist() == [127.0, 64.0, -64.0, -127.0]
    assert a[0, 0] == 2.0 and a[0, 1] == 0.0 and bool(a[0, 2].isnan())
    assert q[0, 64:].abs().sum() == 0


def test_reference_int4_covers_its_range():
    W = torch.tensor([[-7.5, 7.5] + [0.5] * 30, [0.0] * 32]).bfloat16()
    q, s, z = ref.int4(W, 32, True)
    assert s[0, 0] == 1.0 and z[0, 0] == 8 and q[0, :3].tolist() == [0, 15, 9]
    assert s[1, 0] == 0.0 and z[1, 0] == 0 and q[1].max() == 0
    q, s, z = ref.int4(W[:1], 32, False)
    assert z[0, 0] == 8 and q[0, :2].tolist() == [1, 15]


def test_reference_adapter_gradients_against_differences():
    torch.manual_seed(1)
    x, gh, A, B = (torch.randn(*s, dtype=torch.float64) for s in ((7, 64), (7, 5), (3, 64), (5, 3)))
    ga, gb, *_ = ref.lora_grads(x, gh, A, B, 0.5)
    loss = lambda A, B: float((gh * (0.5 * (x @ A.t()) @ B.t())).sum())  # noqa: E731
    for g, P_, i in ((ga, A, (1, 9)), (gb, B, (4, 2))):
        e = torch.zeros_like(P_)
        e[i] = 1e-6
        hi = loss(A + e, B) if P_ is A else loss(A, B + e)
        lo = loss(A - e, B) if P_ is A else loss(A, B - e)
        assert abs((hi - lo) / 2e-6 - float(g[i])) < 1e-6 * max(1.0, abs(float(g[i])))


def test_reference_swiglu_gradient_against_differences():
    torch.manual_seed(0)
    g, u, dy = (torch.randn(200, dtype=torch.float64) * 3 for _ in range(3))
    dg, du = ref.swiglu_grads(g, u, dy)
    e = 1e-6
    ng = (ref.swiglu(g + e, u) - ref.swiglu(g - e, u)) / (2 * e) * dy
    nu = (ref.swiglu(g, u + e) - ref.swiglu(g, u - e)) / (2 * e) * dy
    assert torch.allclose(dg, ng, rtol=1e-6, atol=1e-8) and torch.allclose(du, nu, rtol=1e-6, atol=1e-8)
