"""The 8-bit activations, the SwiGLU over them and the 4-bit integer weights on the GPU against plain 64-bit
forms (lowbit_ref).

Tolerances. A bf16 result is off by half a step, 2^-8 of its value, from the rounding, plus what the fp32
arithmetic before it is off; that part is derived at each test. Codes are compared for equality."""
import threading

import pytest
import torch

import lowbit_ref as ref
from bit_nf4_quantized_25_b200 import binding as qb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = "cuda"
BF = torch.bfloat16
TINY = 2.0 ** -133  # the smallest bf16 step: what a result near zero may be off by


def rand(*shape, std=1.0, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(BF)


def within(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound)[bad].max()):.3g} x"


def guarded(numel, dtype, fill):
    """A buffer of numel elements between two guards of 64; (whole, middle)."""
    whole = torch.full((numel + 128,), fill, dtype=dtype, device=DEV)
    return whole, whole[64:64 + numel]


def guards_kept(whole, fill):
    return bool((whole[:64] == fill).all()) and bool((whole[-64:] == fill).all())


# ------------------------------------------------------------------ activations in 8 bits

def check_act8(x):
    q, a = ref.act8(x)
    got = qb.act8_quantize(x)
    assert torch.equal(got.absmax.double().isnan(), a.isnan())
    assert torch.equal(got.absmax.double().nan_to_num(-1.0), a.nan_to_num(-1.0))
    assert torch.equal(got.codes.double(), q), "codes"
    back = qb.act8_dequantize(got)
    want = ref.act8_values(got.codes, got.absmax)
    assert torch.equal(back.isnan(), want.isnan())
    # s = a / 127 and q s are rounded to fp32 (2^-24 each, or a step of 2^-149 below its normal range), then bf16
    within(back.nan_to_num(0.0), want.nan_to_num(0.0), want.nan_to_num(0.0).abs() * (ref.HALF_STEP + 2.0 ** -22) + TINY)
    return got


@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 192), (7, 4096), (33, 64 * 37), (129, 11008), (2, 28672)])
def test_act8_shapes(rows, cols):
    check_act8(rand(rows, cols, seed=rows))


def test_act8_every_significand_against_every_absmax():
    # blocks whose largest value has each of the 128 significands, with every bf16 value down to 2^-10 of it, at
    # ordinary, largest, smallest normal, subnormal and switch-over (2^-100) magnitudes
    for e in (0x3f80, 0x7f00, 0x0080, 0x0100, 0x0d80, 0x0d00, 0x0e00, 0x0500):
        a = torch.arange(e, e + 128, dtype=torch.int32, device=DEV)
        low = max(e - 10 * 128, 0)
        m = torch.arange(low, e + 128, dtype=torch.int32, device=DEV)
        m = torch.cat([m, torch.zeros((-m.numel()) % 63, dtype=torch.int32, device=DEV)]).reshape(-1, 63)
        v = m.unsqueeze(0).expand(128, -1, -1).reshape(-1, 63)
        top = a.unsqueeze(1).expand(-1, m.shape[0]).reshape(-1, 1)
        v = torch.minimum(v, top)
        sign = (torch.arange(63, device=DEV, dtype=torch.int32) % 2) << 15
        blocks = torch.cat([top, v | sign], 1)
        x = blocks.to(torch.int16).view(BF)
        check_act8(x)
    # every subnormal against every subnormal absmax
    a = torch.arange(1, 128, dtype=torch.int32, device=DEV).reshape(-1, 1)
    v = torch.arange(126, dtype=torch.int32, device=DEV).reshape(1, -1).expand(127, -1)
    v = torch.minimum(v, a).reshape(127, 2, 63)
    x = torch.cat([a.unsqueeze(1).expand(-1, 2, -1), v], 2).reshape(-1, 64).to(torch.int16).view(BF)
    check_act8(x)


def test_act8_nan_infinity_and_zero_blocks():
    x = rand(4, 320, seed=3)
    x[0, 5] = float("nan")
    x[1, 64 * 3 + 63] = float("inf")
    x[2, 64] = float("-inf")
    x[3, :64] = 0.0
    x[3, 64:128] = -0.0
    got = check_act8(x)
    back = qb.act8_dequantize(got)
    assert int(back.isnan().any(1).sum()) == 3 and int(back.isnan().sum()) == 3 * 64
    assert bool((back[3, :128] == 0).all())


def test_act8_writes_only_its_buffers_and_into_those_given():
    x = rand(5, 64 * 9, seed=4)
    n = x.numel()
    cw, c = guarded(n, torch.int8, 77)
    aw, a = guarded(n // 64, BF, 3.0)
    a8 = qb.Act8(5, 64 * 9, c.view(5, -1), a.view(5, -1))
    assert qb.act8_quantize(x, out=a8) is a8
    ow, o = guarded(n, BF, 5.0)
    assert qb.act8_dequantize(a8, out=o.view(5, -1)).data_ptr() == o.data_ptr()
    assert guards_kept(cw, 77) and guards_kept(aw, 3.0) and guards_kept(ow, 5.0)
    assert torch.equal(o.view(5, -1), qb.act8_dequantize(qb.act8_quantize(x)))


def test_act8_rows_taken_out_of_a_longer_one():
    # a row slice of codes and absmax is an activation of its own (absmax then starts on any 2-byte boundary)
    x = rand(6, 192, seed=5)
    a = qb.act8_quantize(x)
    part = qb.Act8(4, 192, a.codes[1:5], a.absmax[1:5])
    assert part.absmax.data_ptr() % 4 != 0
    assert torch.equal(qb.act8_dequantize(part), qb.act8_dequantize(a)[1:5])


def test_act8_beyond_32_bit_offsets():
    rows, cols = 2 ** 31 // 8192 + 3, 8192  # the last rows start past 2^31 values
    x = torch.zeros(rows, cols, dtype=BF, device=DEV)
    x[-3:] = rand(3, cols, seed=6)
    a = qb.act8_quantize(x)
    q, top = ref.act8(x[-3:])
    assert torch.equal(a.codes[-3:].double(), q) and torch.equal(a.absmax[-3:].double(), top)
    assert int(a.codes[:-3].count_nonzero()) == 0
    y = qb.act8_dequantize(a, out=x)
    assert torch.equal(y[-3:], qb.act8_dequantize(qb.Act8(3, cols, a.codes[-3:], a.absmax[-3:])))


# ---------------------------------------------------------------------------- SwiGLU

def check_swiglu(gate, up, dy):
    y, g8, u8 = qb.swiglu_act8_fwd(gate, up)
    for a, x in ((g8, gate), (u8, up)):
        q, top = ref.act8(x)
        assert torch.equal(a.codes.double(), q) and torch.equal(a.absmax.double(), top)
    # exp2 of a rounded argument: relative error of exp(-g) at most (2 + 1.2 |g|) 2^-23, of 1 / (1 + exp) and the
    # products 4 units of 2^-23 more. The quotient reads 0 where 1 + exp(-g) is above 2^126, that is below 2^-118.
    g, u = gate.double(), up.double()
    eta = (6.0 + 1.2 * g.abs()) * 2.0 ** -23
    want = ref.swiglu(g, u)
    within(y, want, want.abs() * (ref.HALF_STEP + 1.01 * eta) + (1.0 + u.abs()) * 2.0 ** -118, "y")

    gg, gu, y8 = qb.swiglu_act8_bwd(g8, u8, dy)
    g, u, d = ref.act8_values(g8.codes, g8.absmax), ref.act8_values(u8.codes, u8.absmax), dy.double()
    eta = (8.0 + 1.2 * g.abs()) * 2.0 ** -23  # two roundings more, of g and u read back
    dg, du = ref.swiglu_grads(g, u, d)
    sig = 1.0 / (1.0 + torch.exp(-g))
    floor = (1.0 + u.abs()) * (1.0 + d.abs()) * 2.0 ** -118
    # 1 + g (1 - sigma) cancels: it is off by (1 + |g|) 2^-22 + |g| sigma eta whatever its value
    slack = (d * u * sig).abs() * ((1.0 + g.abs()) * 2.0 ** -22 + g.abs() * sig * eta)
    within(gg, dg, dg.abs() * (ref.HALF_STEP + 1.01 * eta) + 1.01 * slack + floor, "grad_gate")
    within(gu, du, du.abs() * (ref.HALF_STEP + 1.01 * eta) + floor, "grad_up")
    # y again: rounded to bf16, then within a / 254 of that, a the block's (rounded) largest
    want = ref.swiglu(g, u)
    back = ref.act8_values(y8.codes, y8.absmax)
    top = want.abs().reshape(want.shape[0], -1, 64).amax(-1, keepdim=True).expand(-1, -1, 64).reshape(want.shape)
    rounding = want.abs() * (ref.HALF_STEP + 1.01 * eta) + (1.0 + u.abs()) * 2.0 ** -118
    within(back, want, rounding + top * 1.01 / 254.0 + 2.0 ** -118, "y8")
    a, b, none = qb.swiglu_act8_bwd(g8, u8, dy, recompute=False)
    assert none is None and torch.equal(a, gg) and torch.equal(b, gu)


@pytest.mark.parametrize("rows,cols", [(1, 64), (1, 11008), (5, 192), (77, 64 * 43), (130, 11008)])
def test_swiglu(rows, cols):
    check_swiglu(rand(rows, cols, std=1.5, seed=1), rand(rows, cols, seed=2), rand(rows, cols, seed=3))


def test_swiglu_over_the_whole_range_of_gates():
    g = torch.linspace(-200, 200, 64 * 64, device=DEV).to(BF).reshape(8, -1)
    check_swiglu(g, rand(8, 512, std=4.0, seed=8), rand(8, 512, seed=9))


def test_swiglu_gradient_against_differences():
    # the derivative at the kept values, from the forward kernel's own formula at neighbouring gates
    gate, up, dy = rand(4, 256, std=1.5, seed=1), rand(4, 256, seed=2), rand(4, 256, seed=3)
    _, g8, u8 = qb.swiglu_act8_fwd(gate, up)
    gg, gu, _ = qb.swiglu_act8_bwd(g8, u8, dy)
    g, u = qb.act8_dequantize(g8).double(), qb.act8_dequantize(u8).double()
    e = 1e-5
    dg = (ref.swiglu(g + e, u) - ref.swiglu(g - e, u)) / (2 * e) * dy.double()
    du = (ref.swiglu(g, u + e) - ref.swiglu(g, u - e)) / (2 * e) * dy.double()
    # g and u are read back in bf16 here and in fp32 by the kernel: half a step of each moves the gradients by up to
    # 2^-8 (|g f'' u| + |f' u|) |dy|, with |g f''| <= 0.6 + ... <= 1 and |f'| <= 1.1
    slack = 2.0 ** -8 * dy.double().abs() * (2.2 * u.abs() + 1.1 * g.abs())
    within(gg, dg, dg.abs() * 2.0 ** -7 + slack + 1e-6)
    within(gu, du, du.abs() * 2.0 ** -7 + slack + 1e-6)


def test_swiglu_of_one_tensor_as_gate_and_up():
    x, dy = rand(5, 192, seed=1), rand(5, 192, seed=2)
    y, g8, u8 = qb.swiglu_act8_fwd(x, x)
    assert torch.equal(y, qb.swiglu_act8_fwd(x, x.clone())[0]) and torch.equal(g8.codes, u8.codes)
    got = qb.swiglu_act8_bwd(g8, g8, dy)
    want = qb.swiglu_act8_bwd(g8, u8, dy)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2].codes, want[2].codes)


def test_swiglu_nan_block_reaches_the_gradients():
    gate, up, dy = rand(2, 128, seed=1), rand(2, 128, seed=2), rand(2, 128, seed=3)
    gate[1, 70] = float("inf")
    y, g8, u8 = qb.swiglu_act8_fwd(gate, up)
    gg, gu, y8 = qb.swiglu_act8_bwd(g8, u8, dy)
    bad = torch.zeros(2, 128, dtype=torch.bool, device=DEV)
    bad[1, 64:] = True
    assert torch.equal(gg.isnan(), bad) and torch.equal(gu.isnan(), bad)
    assert torch.equal(qb.act8_dequantize(y8).isnan(), bad)


# ------------------------------------------------------------------- adapter gradients

def check_grads(x8, gh, A, B, alpha, keep=None, dropout=None, **kw):
    M, n, k, r = gh.shape[0], gh.shape[1], A.shape[1], A.shape[0]
    ga, gb = qb.qlora_lora_grads_act8(x8, gh, A, B, alpha, dropout=dropout, **kw)
    x, s = ref.act8_values(x8.codes, x8.absmax), alpha / r
    if keep is not None:
        x, s = x * keep, s / (1.0 - dropout[0])
    wa, wb, sa, sb = ref.lora_grads(x, gh.double(), A.double(), B.double(), s)
    # In units of the sum of the terms' sizes: t (u) is a chain of fp32 additions, 4 of the tensor core and one fma for
    # 64 features, and 8 over the cluster (2^-23 each); three bf16 terms leave 2^-24; the products over tokens are a chain
    # of 3 for 16 tokens and 10 over the CTA and cluster (2^-23 each); s and a / 127 2^-23 each.
    def unit(features):
        return ((5 * features / 64 + 8) + (3 * (M / 16 + 1) + 10) + 5) * 2.0 ** -23
    within(ga, wa, sa * unit(n) + 1e-30, "grad_A")
    within(gb, wb, sb * unit(k) + 1e-30, "grad_B")
    return ga, gb


def grad_inputs(M, n, k, r, seed=0):
    x8 = qb.act8_quantize(rand(M, k, seed=seed))
    return x8, rand(M, n, seed=seed + 1), rand(r, k, std=0.01, seed=seed + 2), rand(n, r, std=0.01, seed=seed + 3)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 100, 127, 128, 129, 300, 1000])
def test_grads_tokens(M):
    check_grads(*grad_inputs(M, 200, 192, 16, seed=M), 32.0)


@pytest.mark.parametrize("r", [1, 3, 8, 13, 16, 17, 32, 33, 64, 65, 100, 128, 256])
def test_grads_ranks(r):
    check_grads(*grad_inputs(70, 136, 320, r, seed=r), 2.0 * r)


@pytest.mark.parametrize("n,k", [(1, 64), (7, 64), (8, 128), (63, 448), (255, 256), (257, 320), (1000, 64 * 21),
                                 (4096, 4096), (11008, 4096), (4096, 11008), (4097, 64 * 17)])
def test_grads_shapes(n, k):
    check_grads(*grad_inputs(150, n, k, 16, seed=n), 32.0)


@pytest.mark.parametrize("n,k,r", [(4096, 4096, 16), (1028, 1024, 64), (1031, 1024, 24)])
def test_grads_long_batches(n, k, r):
    check_grads(*grad_inputs(4099, n, k, r, seed=n), 32.0)


# from 1025 tokens on the kernels for long batches run whatever the rest is
@pytest.mark.parametrize("M", [1024, 1025, 1056, 1087, 1151, 1152, 1153])
def test_grads_long_batch_tokens(M):
    check_grads(*grad_inputs(M, 200, 192, 16, seed=M), 32.0)


@pytest.mark.parametrize("r", [1, 3, 8, 13, 16, 17, 32, 33, 64, 65, 100, 128, 256])
def test_grads_long_batch_ranks(r):
    check_grads(*grad_inputs(1070, 136, 320, r, seed=r), 2.0 * r)


@pytest.mark.parametrize("n,k", [(1, 64), (7, 64), (8, 128), (63, 448), (255, 256), (257, 320), (1000, 64 * 21), (4097, 64 * 17)])
def test_grads_long_batch_shapes(n, k):
    check_grads(*grad_inputs(1150, n, k, 16, seed=n), 32.0)


def test_grads_long_batch_dropout(oracle):
    M, n, k, r = 1100, 200, 320, 24
    p, seed, offset = 0.25, 1234567890123, 2 ** 33 + 1
    keep = torch.from_numpy(oracle.dropout_keep(seed, offset, p, M, k)).to(DEV)
    check_grads(*grad_inputs(M, n, k, r), 8.0, keep=keep.double(), dropout=(p, seed, offset))


def test_grads_long_batch_is_reproducible_and_stays_inside_its_buffers():
    M, n, k, r = 1130, 205, 192, 13
    x8, gh, A, B = grad_inputs(M, n, k, r)
    aw, a = guarded(r * k, torch.float32, 3.0)
    bw, b = guarded(n * r, torch.float32, 5.0)
    need = qb.lora_grads_act8_workspace_size(M, n, r)
    ww = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
    w = ww[256:256 + need]
    first = check_grads(x8, gh, A, B, 8.0, grad_A=a.view(r, k), grad_B=b.view(n, r), workspace=w)
    again = qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    assert guards_kept(aw, 3.0) and guards_kept(bw, 5.0)
    assert bool((ww[:256] == 77).all()) and bool((ww[-256:] == 77).all())


def test_grads_70b_layer():
    check_grads(*grad_inputs(1030, 28672, 8192, 64, seed=1), 16.0)


@pytest.mark.parametrize("offset", [0, 3, 2 ** 33 + 1])
@pytest.mark.parametrize("r", [4, 40])
def test_grads_dropout(oracle, offset, r):
    M, n, k = 37, 50, 192
    p, seed = 0.25, 1234567890123
    x8, gh, A, B = grad_inputs(M, n, k, r)
    keep = torch.from_numpy(oracle.dropout_keep(seed, offset, p, M, k)).to(DEV)
    assert 0.6 < float(keep.double().mean()) < 0.9
    ga, gb = check_grads(x8, gh, A, B, 8.0, keep=keep.double(), dropout=(p, seed, offset))
    plain = qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0)
    off = qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0, dropout=(0.0, seed, offset))
    assert all(torch.equal(a, b) for a, b in zip(plain, off)) and not torch.equal(ga, plain[0])


def test_grads_agree_with_the_16_bit_entry_point():
    # an input whose values an 8-bit block holds exactly: the same gradients as from bf16, to that call's own 1e-2
    M, n, k, r = 200, 320, 256, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.randint(-127, 128, (M, k), device=DEV, generator=g).to(BF)
    x[:, ::64] = 127.0
    x8 = qb.act8_quantize(x)
    assert torch.equal(qb.act8_dequantize(x8), x)
    _, gh, A, B = grad_inputs(M, n, k, r)
    for d in (None, (0.1, 7, 2)):
        for a, b in zip(qb.qlora_lora_grads_act8(x8, gh, A, B, 32.0, dropout=d),
                        qb.qlora_lora_grads(x, gh, A, B, 32.0, dropout=d)):
            a, b = a.double(), b.double()
            within(a, b, 1e-2 * b.abs() + 1e-2 * b.square().mean().sqrt())


def test_grads_are_reproducible_and_stay_inside_their_buffers():
    M, n, k, r = 130, 205, 192, 13
    x8, gh, A, B = grad_inputs(M, n, k, r)
    aw, a = guarded(r * k, torch.float32, 7.0)
    bw, b = guarded(n * r, torch.float32, 7.0)
    need = qb.lora_grads_act8_workspace_size(M, n, r)
    whole = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
    first = qb.qlora_lora_grads_act8(x8, gh, A, B, 26.0, grad_A=a.view(r, k), grad_B=b.view(n, r),
                                     workspace=whole[256:256 + need])
    assert guards_kept(aw, 7.0) and guards_kept(bw, 7.0)
    assert bool((whole[:256] == 77).all()) and bool((whole[256 + need:] == 77).all())
    for _ in range(3):
        again = qb.qlora_lora_grads_act8(x8, gh, A, B, 26.0)
        assert all(torch.equal(u, v) for u, v in zip(first, again))


def test_grads_empty_sides():
    x8, gh, A, B = grad_inputs(0, 40, 128, 8)
    ga, gb = qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0)
    assert int(ga.count_nonzero()) == 0 and int(gb.count_nonzero()) == 0
    x8, _, A, _ = grad_inputs(5, 40, 128, 8)
    ga, gb = qb.qlora_lora_grads_act8(x8, rand(5, 0), A, rand(0, 8), 8.0)
    assert gb.shape == (0, 8) and int(ga.count_nonzero()) == 0


def test_grads_nan_block_and_zero_blocks():
    M, n, k, r = 40, 72, 192, 8
    x = rand(M, k, seed=1)
    x[:, 64:128] = 0.0
    x8 = qb.act8_quantize(x)
    _, gh, A, B = grad_inputs(M, n, k, r)
    ga, _ = check_grads(x8, gh, A, B, 8.0)
    assert int(ga[:, 64:128].count_nonzero()) == 0
    x[7, 3] = float("nan")
    ga, gb = qb.qlora_lora_grads_act8(qb.act8_quantize(x), gh, A, B, 8.0)
    assert bool(gb.isnan().all()) and bool(ga[:, :64].isnan().all()) and not bool(ga[:, 64:].isnan().any())


def test_grads_against_differences():
    # the loss is sum(grad_h * s B A x) over the values read back; moved along one entry of A and of B
    M, n, k, r = 33, 48, 128, 8
    x8, gh, A, B = grad_inputs(M, n, k, r)
    ga, gb = qb.qlora_lora_grads_act8(x8, gh, A, B, 16.0)
    x, g = ref.act8_values(x8.codes, x8.absmax), gh.double()
    loss = lambda A, B: float((g * (2.0 * (x @ A.t()) @ B.t())).sum())  # noqa: E731
    for j, i in ((0, 0), (7, 127), (3, 70)):
        e = torch.zeros(r, k, dtype=torch.float64, device=DEV)
        e[j, i] = 1e-3
        d = (loss(A.double() + e, B.double()) - loss(A.double() - e, B.double())) / 2e-3  # linear in A: exact
        assert abs(d - float(ga[j, i])) <= 1e-4 * float(ga.abs().max())
    for i, j in ((0, 0), (47, 7), (20, 3)):
        e = torch.zeros(n, r, dtype=torch.float64, device=DEV)
        e[i, j] = 1e-3
        d = (loss(A.double(), B.double() + e) - loss(A.double(), B.double() - e)) / 2e-3
        assert abs(d - float(gb[i, j])) <= 1e-4 * float(gb.abs().max())


# ------------------------------------------------------------------- 4-bit integers

@pytest.mark.parametrize("n,k", [(1, 128), (3, 384), (17, 1280), (100, 4096), (33, 11008)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [True, False])
def test_int4_quantize(n, k, group, zero):
    W = rand(n, k, std=0.02, seed=n)
    check_int4(W, group, zero)


def check_int4(W, group, zero):
    q, s, z = ref.int4(W, group, zero)
    w = qb.int4_quantize(W, group=group, zero_point=zero)
    assert torch.equal(w.scale.cpu().view(torch.int16), s.view(torch.int16)), "scale"
    if zero:
        assert torch.equal(w.zero_point.cpu().long(), torch.from_numpy(z)), "zero point"
    else:
        assert w.zero_point is None
    assert torch.equal(ref.int4_unpack(w.codes).cpu().long(), torch.from_numpy(q)), "codes"
    want = ref.int4_values(w.codes, w.scale, w.zero_point, group)
    # s (q - z) is exact in fp32: one rounding
    assert torch.equal(qb.int4_dequantize(w).view(torch.int16), want.float().to(BF).view(torch.int16))
    return w


def test_int4_halves_constants_and_extremes():
    W = torch.zeros(16, 128)
    W[0] = torch.arange(128) / 16.0 - 4.0  # many halves of a step
    W[1] = torch.arange(128) % 15 - 7.0
    W[2] = (torch.arange(128) % 29 - 14.0) / 2.0
    W[3] = 0.375
    W[4] = -0.375
    W[5, 7] = 3.0
    W[6, 9] = -3.0
    W[7] = torch.where(torch.arange(128) % 2 == 0, 3.3e38, -3.3e38)  # max - min overflows fp32
    W[8] = torch.arange(128) * 2.0 ** -133
    W[9] = (torch.arange(128) - 64) * 2.0 ** -110
    W[10] = torch.arange(128) * 2.0 ** -104
    W[11, 0] = 2.0 ** -133
    W[12] = torch.linspace(1.0, 2.0, 128)
    W[13] = -torch.linspace(1.0, 2.0, 128)
    W[14] = torch.randn(128, generator=torch.Generator().manual_seed(0)) * 2.0 ** -100
    W = W.to(BF).to(DEV)
    for group in (32, 64, 128):
        check_int4(W[[0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 11, 12, 13, 14, 15]].contiguous(), group, True)
        check_int4(W[[0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 11, 12, 13, 14, 15]].contiguous(), group, False)
        w = qb.int4_quantize(W[7:8].contiguous(), group=group)
        back = qb.int4_dequantize(w).double()
        step = 2 * 3.3e38 / 15
        # half a step of the code (+-7.5 steps is a half: one end takes 7, the other 8 steps), 8 times the rounding of
        # the step to bf16 (8 * 2^-8), and the rounding of up to 8 steps to bf16 (8 * 2^-8): 0.5 + 0.0625
        assert bool(back.isfinite().all()) and float((back - W[7:8].double()).abs().max()) <= 0.5625 * step


@pytest.mark.parametrize("exponent", [0, 100, 119, -55, -57, -100, -120])
def test_int4_every_pair_of_range_significands(exponent):
    # groups of 64 from -b to a for each of the 128 significands of a and of b (a sixteenth, half, twice and as large), with
    # weights at multiples of half a step; the exponents lie on both sides of what is an ordinary range
    g = torch.Generator().manual_seed(exponent % 1000)
    a = (1.0 + torch.arange(128) / 128.0).view(-1, 1).expand(128, 128)
    b = (1.0 + torch.arange(128) / 128.0).view(1, -1) * torch.tensor([1.0, 0.0625, 0.5, 2.0])[torch.randint(0, 4, (128, 128), generator=g)]
    half = ((a + b) / 30.0).unsqueeze(-1)
    low = -(b.unsqueeze(-1) / half).floor()
    k = low + (torch.rand(128, 128, 62, generator=g) * ((a.unsqueeze(-1) / half).floor() - low)).round()
    W = torch.cat([a.unsqueeze(-1), -b.unsqueeze(-1), (k * half).clamp(-b.unsqueeze(-1), a.unsqueeze(-1))], -1)
    W = (W.double() * 2.0 ** exponent).reshape(128, -1).to(BF).to(DEV)
    check_int4(W, 64, True)
    check_int4(W, 64, False)


def test_int4_writes_only_its_buffers():
    n, k, group = 5, 384, 64
    W = rand(n, k, std=0.02, seed=1)
    cw, c = guarded(n * k // 2, torch.uint8, 200)
    sw, s = guarded(n * k // group, BF, 3.0)
    zw, z = guarded(n * k // group, torch.uint8, 99)
    w = qb.Int4Weight(n, k, group, c.view(n, -1), s.view(n, -1), z.view(n, -1))
    qb.int4_quantize(W, out=w)
    hw, h = guarded(3 * n, BF, 7.0)
    qb.int4_linear_fwd(w, rand(3, k, seed=2), out=h.view(3, n))
    assert guards_kept(cw, 200) and guards_kept(sw, 3.0) and guards_kept(zw, 99) and guards_kept(hw, 7.0)
    other = qb.int4_quantize(W, group=group)
    assert torch.equal(other.codes, w.codes) and torch.equal(other.scale, w.scale)


def random_int4(n, k, group, zero, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), device=DEV, generator=g, dtype=torch.uint8)
    scale = (0.002 + 0.01 * torch.rand(n, k // group, device=DEV, generator=g)).to(BF)
    z = torch.randint(0, 16, (n, k // group), device=DEV, generator=g, dtype=torch.uint8) if zero else None
    return qb.Int4Weight(n, k, group, codes, scale, z)


def check_linear(w, x):
    h = qb.int4_linear_fwd(w, x)
    W = ref.int4_values(w.codes, w.scale, w.zero_point, w.group)
    want, size = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    # products are exact; a group's sum is 8 accumulations of the tensor core (2^-22 of the sum of sizes each at
    # most), the groups' sums are joined by at most 48 fp32 additions in a row per warp and 19 over the parts of k
    # (2^-24 each): below 2^-17
    within(h, want, want.abs() * ref.HALF_STEP + size * 2.0 ** -17 + TINY)
    return h


@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 17, 40, 64])
@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, True)])
def test_int4_linear_tokens(M, group, zero):
    check_linear(random_int4(200, 1280, group, zero, seed=M), rand(M, 1280, seed=M))


@pytest.mark.parametrize("n,k", [(1, 128), (15, 128), (16, 256), (17, 384), (1001, 640), (4096, 4096), (11008, 4096),
                                 (4096, 11008), (130, 28672)])
@pytest.mark.parametrize("group,zero", [(32, False), (64, True), (128, False)])
def test_int4_linear_shapes(n, k, group, zero):
    check_linear(random_int4(n, k, group, zero, seed=n), rand(3, k, seed=k))


@pytest.mark.parametrize("k,group", [(64, 32), (64, 64), (192, 64), (192, 32)])
def test_int4_linear_fewer_groups_than_warps(k, group):
    check_linear(random_int4(40, k, group, True, seed=1), rand(2, k, seed=2))


@pytest.mark.parametrize("n,k,M", [(80000, 256, 2), (7700, 24576, 3), (7700, 24576, 16), (48, 36864, 12), (16, 65536, 17)])
def test_int4_linear_many_rounds_and_long_rows(n, k, M):
    check_linear(random_int4(n, k, 64, True, seed=n), rand(M, k, seed=k))


def test_int4_linear_outliers_and_non_finite_tokens():
    w = random_int4(64, 512, 128, True, seed=1)
    x = rand(4, 512, seed=2)
    x[1, 17] = 3.0e4
    x[2, :] = 3.0e-39  # subnormal activations
    check_linear(w, x)
    x[3, 100] = float("nan")
    h = qb.int4_linear_fwd(w, x)
    assert bool(h[3].isnan().all()) and not bool(h[:3].isnan().any())


@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_linear_infinite_activations(group):
    w = random_int4(64, 512, group, True, seed=1)
    x = rand(3, 512, seed=2)
    x[0, 17], x[2, 511] = float("inf"), float("-inf")
    h = qb.int4_linear_fwd(w, x).double()
    want = x.double() @ ref.int4_values(w.codes, w.scale, w.zero_point, group).t()
    assert torch.equal(h.isnan(), want.isnan()) and torch.equal(h.isinf(), want.isinf())
    assert torch.equal(h[h.isinf()], want[want.isinf()])


def test_int4_linear_tokens_do_not_depend_on_their_neighbours():
    w = random_int4(300, 1024, 64, True, seed=1)
    x = rand(16, 1024, seed=2)
    h = qb.int4_linear_fwd(w, x)
    for m in (1, 5, 8, 11):
        assert torch.equal(qb.int4_linear_fwd(w, x[:m]), h[:m])
    assert torch.equal(qb.int4_linear_fwd(w, x), h)


@pytest.mark.parametrize("n,k,group", [(4096, 4096, 128), (688, 11008, 32), (64, 36864, 64)])
def test_int4_linear_token_alone_or_in_a_batch(n, k, group):
    w = random_int4(n, k, group, True, seed=n)
    x = rand(33, k, seed=3)
    h = qb.int4_linear_fwd(w, x)
    for a, b in ((0, 1), (7, 9), (20, 33)):
        assert torch.equal(qb.int4_linear_fwd(w, x[a:b]), h[a:b])


def test_int4_empty():
    w = random_int4(64, 512, 128, True)
    assert qb.int4_linear_fwd(w, rand(0, 512)).shape == (0, 64)
    e = qb.int4_quantize(torch.empty(0, 256, dtype=BF, device=DEV))
    assert qb.int4_dequantize(e).shape == (0, 256)
    z = qb.Int4Weight.empty(5, 0, 64)
    assert bool((qb.int4_linear_fwd(z, rand(2, 0)) == 0).all())


# --------------------------------------------------------------------- streams, graphs

def test_calls_on_another_stream_and_in_a_graph():
    x, gate, up, dy = (rand(9, 640, seed=s) for s in range(4))
    W, xs = rand(96, 640, std=0.02, seed=5), rand(4, 640, seed=6)
    A, B = rand(8, 640, seed=7), rand(640, 8, seed=8)

    def step(stream=None):
        a = qb.act8_quantize(x, stream=stream)
        y, g8, u8 = qb.swiglu_act8_fwd(gate, up, stream=stream)
        gg, gu, y8 = qb.swiglu_act8_bwd(g8, u8, dy, stream=stream)
        ga, gb = qb.qlora_lora_grads_act8(a, up, A, B, 8.0, stream=stream, dropout=(0.1, 5, 0))
        w = qb.int4_quantize(W, stream=stream)
        h = qb.int4_linear_fwd(w, xs, stream=stream)
        return (qb.act8_dequantize(a, stream=stream), y, gg, gu, ga, gb, qb.act8_dequantize(y8, stream=stream),
                qb.int4_dequantize(w, stream=stream), h)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in (20, 30):
        for i, t in enumerate((x, gate, up, dy, W, xs)):
            t.copy_(rand(*t.shape, std=0.02 if t is W else 1.0, seed=seed + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


@pytest.mark.parametrize("M,n,k,r,dropout", [(1200, 1001, 448, 70, None), (1300, 512, 512, 16, (0.1, 5, 3)), (200, 1001, 448, 70, None), (40, 130, 192, 90, None)])
def test_grads_in_a_graph(M, n, k, r, dropout):
    x8, gh, A, B = grad_inputs(M, n, k, r)
    ws = torch.empty(qb.lora_grads_act8_workspace_size(M, n, r), dtype=torch.uint8, device=DEV)
    call = lambda: qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0, workspace=ws, dropout=dropout)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call()
    for seed in (20, 30):
        y8, *rest = grad_inputs(M, n, k, r, seed=seed)
        for t, v in zip((x8.codes, x8.absmax, gh, A, B), (y8.codes, y8.absmax, *rest)):
            t.copy_(v)
        graph.replay()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(kept, call()))


def test_calls_side_by_side_on_two_streams():
    sides = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        x8, gh, A, B = grad_inputs(512, 1024, 1024, 16, seed=10 * i)
        w = random_int4(4096, 4096, 64, True, seed=i)
        sets.append((x8, gh, A, B, w, rand(16, 4096, seed=i), rand(64, 1024, seed=i), rand(64, 1024, seed=i + 5)))

    def run(x8, gh, A, B, w, x, gate, up):
        y, g8, u8 = qb.swiglu_act8_fwd(gate, up)
        return (*qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0), qb.int4_linear_fwd(w, x), y, qb.swiglu_act8_bwd(g8, u8, up)[0])

    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i].append(run(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


def test_host_threads_with_a_stream_each():
    x8, gh, A, B = grad_inputs(1100, 512, 512, 16)
    w, x = random_int4(4096, 4096, 64, True, seed=1), rand(16, 4096, seed=2)

    def run():
        return (qb.int4_linear_fwd(w, x), *qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0), qb.act8_quantize(x).codes)

    want = run()
    torch.cuda.synchronize()
    same = []

    def work():
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = [run() for _ in range(20)]
        side.synchronize()
        same.append(all(torch.equal(p, q) for g in got for p, q in zip(g, want)))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True] * 3


@pytest.mark.parametrize("rows,cols", [(3, 192), (700, 4096)])
def test_back_to_back_launches_see_what_the_one_before_wrote(rows, cols):
    # one set of buffers in turn: a kernel may be set up, but not read or write, before the one before it is done
    xs = [rand(rows, cols, std=0.02 * (i + 1), seed=i) for i in range(8)]
    W = [rand(256, cols, std=0.02, seed=i) for i in range(8)]
    want = [(qb.act8_dequantize(qb.act8_quantize(x)), qb.int4_linear_fwd(qb.int4_quantize(w, group=64), x[:3]),
             qb.int4_dequantize(qb.int4_quantize(w, group=64))) for x, w in zip(xs, W)]
    torch.cuda.synchronize()
    a, w = qb.Act8.empty(rows, cols), qb.Int4Weight.empty(256, cols, 64)
    got = []
    for x, v in zip(xs * 4, W * 4):
        qb.act8_quantize(x, out=a)
        y = qb.act8_dequantize(a)
        qb.int4_quantize(v, out=w)
        got.append((y, qb.int4_linear_fwd(w, x[:3]), qb.int4_dequantize(w)))
    assert all(torch.equal(p, q) for i, g in enumerate(got) for p, q in zip(g, want[i % 8]))


def test_results_do_not_land_in_memory_that_the_current_stream_still_uses():
    x, w = rand(64, 640, seed=1), random_int4(64, 640, 64, True, seed=2)
    want_a, want_h = qb.act8_quantize(x).codes, qb.int4_linear_fwd(w, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, want in ((lambda: qb.act8_quantize(x, stream=side).codes, want_a),
                       (lambda: qb.int4_linear_fwd(w, x, stream=side), want_h)):
        late = [torch.empty_like(want) for _ in range(4)]
        torch.cuda._sleep(20_000_000)
        for t in late:
            t.zero_()
        del late, t
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_binding_refusals_on_the_gpu():
    x = rand(4, 128)
    a = qb.act8_quantize(x)
    w = random_int4(8, 128, 64, True)
    with pytest.raises(ValueError):
        qb.act8_quantize(x, out=qb.Act8.empty(3, 128))
    with pytest.raises(ValueError):
        qb.act8_dequantize(a, out=torch.empty(4, 128, device=DEV))
    with pytest.raises(ValueError):
        qb.swiglu_act8_fwd(x, x[:, :64])
    with pytest.raises(qb.QNError):
        qb.swiglu_act8_fwd(x, x, out=x)
    with pytest.raises(ValueError):
        qb.swiglu_act8_bwd(a, qb.Act8.empty(4, 64), x)
    with pytest.raises(ValueError):
        qb.swiglu_act8_bwd(a, a, x, y8=qb.Act8.empty(4, 128), recompute=False)
    with pytest.raises(ValueError):
        qb.int4_linear_fwd(w, rand(2, 64))
    with pytest.raises(ValueError):
        qb.int4_linear_fwd(w, rand(2, 128).cpu())
    with pytest.raises(ValueError):
        qb.int4_linear_fwd(w, rand(2, 128), out=torch.empty(2, 9, dtype=BF, device=DEV))
    with pytest.raises(qb.QNError) as e:
        qb.int4_linear_fwd(w, rand(65, 128))
    assert e.value.status == qb.QN_ESHAPE
    with pytest.raises(qb.QNError):
        qb.int4_quantize(rand(4, 128), group=48)


# ------------------------------------------------------------------ the calls together

def test_a_training_step_then_the_merged_layer_decodes():
    """One MLP of a frozen 4-bit base: gate, up and down with adapters, forward and backward with what is kept in 8
    bits, a step on the adapters, the merge, and the merged down projection served from 4-bit integers."""
    M, d, f, r, alpha, lr = 50, 256, 448, 8, 16.0, 0.5
    s = alpha / r
    W = {nm: rand(*sh, std=0.05, seed=i) for i, (nm, sh) in enumerate((("gate", (f, d)), ("up", (f, d)), ("down", (d, f))))}
    w = {nm: qb.nf4_quantize(v) for nm, v in W.items()}
    A = {nm: rand(r, v.shape[1], std=0.05, seed=10 + i) for i, (nm, v) in enumerate(W.items())}
    B = {nm: rand(v.shape[0], r, std=0.05, seed=20 + i) for i, (nm, v) in enumerate(W.items())}
    x, dy = rand(M, d, seed=30), rand(M, d, seed=31)

    x8 = qb.act8_quantize(x)
    gate, up = (qb.qlora_linear_fwd(w[nm], x, A[nm], B[nm], alpha) for nm in ("gate", "up"))
    act, gate8, up8 = qb.swiglu_act8_fwd(gate, up)
    y = qb.qlora_linear_fwd(w["down"], act, A["down"], B["down"], alpha)
    d_act = qb.qlora_linear_bwd_x(w["down"], dy, A["down"], B["down"], alpha)
    d_gate, d_up, act8 = qb.swiglu_act8_bwd(gate8, up8, d_act)
    grads = {"down": qb.qlora_lora_grads_act8(act8, dy, A["down"], B["down"], alpha),
             "gate": qb.qlora_lora_grads_act8(x8, d_gate, A["gate"], B["gate"], alpha),
             "up": qb.qlora_lora_grads_act8(x8, d_up, A["up"], B["up"], alpha)}

    # the same in 64 bits without any rounding of activations
    D = {nm: qb.nf4_dequantize(w[nm]).double() + s * B[nm].double() @ A[nm].double() for nm in W}
    g, u = x.double() @ D["gate"].t(), x.double() @ D["up"].t()
    a = ref.swiglu(g, u)
    da = dy.double() @ D["down"]
    dg, du = ref.swiglu_grads(g, u, da)
    want = {"down": ref.lora_grads(a, dy.double(), A["down"].double(), B["down"].double(), s),
            "gate": ref.lora_grads(x.double(), dg, A["gate"].double(), B["gate"].double(), s),
            "up": ref.lora_grads(x.double(), du, A["up"].double(), B["up"].double(), s)}
    for nm in W:
        for got, exact in zip(grads[nm], want[nm][:2]):
            # 8 bits of a block leave at most 1/254 of its largest, near 1 % of the rms; a gradient mixes a few of these
            assert float((got.double() - exact).norm() / exact.norm()) < 0.05, nm
    assert float((y.double() - a @ D["down"].t()).norm() / (a @ D["down"].t()).norm()) < 0.03

    for nm in W:
        A[nm] = (A[nm].float() - lr * grads[nm][0]).to(BF)
        B[nm] = (B[nm].float() - lr * grads[nm][1]).to(BF)
    merged = qb.qlora_merge_bf16(w["down"], A["down"], B["down"], alpha)
    served = qb.int4_quantize(merged, group=64)
    tok = rand(3, f, seed=40)
    h = qb.int4_linear_fwd(served, tok)
    exact = tok.double() @ qb.int4_dequantize(served).double().t()
    within(h, exact, exact.abs() * 2.0 ** -7 + (tok.double().abs() @ merged.double().abs().t()) * 2.0 ** -7)
    full = tok.double() @ merged.double().t()
    assert float((h.double() - full).norm() / full.norm()) < 0.25  # 4 bits
