"""The 8-bit activations and the 4-bit integer weights on the GPU where their other tests do not reach: weights that are not
finite, gates far below zero, the kernels for few tokens over wide layers, LoRA dropout of long batches at every rank that has
a kernel of its own, buffers of more than 2^31 elements, waits that run out, calls without the compiled marshalling. Compared
with 64-bit forms (lowbit_ref)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import lowbit_ref as ref
from bit_nf4_quantized_25_b200 import binding as qb
from test_lowbit_gpu import BF, DEV, TINY, check_grads, grad_inputs, rand, within

SMS = torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------- 4-bit integers

@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_int4_a_weight_that_is_not_finite_marks_its_group_and_no_other(bad, group, zero):
    n, k = 40, 512
    W = rand(n, k, std=0.02, seed=group)
    clean = qb.int4_quantize(W, group=group, zero_point=zero)
    # row i: the i-th place of a word and of a lane, in a group that moves along the row; row 0 has none
    rows = torch.arange(1, n, device=DEV)
    cols = (rows % (k // group)) * group + rows % group
    W[rows, cols] = bad
    W[9, cols[8] // group * group:cols[8] // group * group + group:2] = float("nan")  # several of them
    w = qb.int4_quantize(W, group=group, zero_point=zero)
    hit = torch.zeros(n, k // group, dtype=torch.bool, device=DEV)
    hit[rows, cols // group] = True
    assert torch.equal(w.scale.isnan(), hit)
    assert torch.equal(w.scale[~hit], clean.scale[~hit])
    q, q0 = (ref.int4_unpack(t.codes).view(n, -1, group) for t in (w, clean))
    assert torch.equal(q[~hit], q0[~hit]), "codes of other groups"
    assert bool((q[hit] == (0 if zero else 8)).all())
    if zero:
        assert torch.equal(w.zero_point[~hit], clean.zero_point[~hit]) and not bool(w.zero_point[hit].any())
    back = qb.int4_dequantize(w)
    wide = hit.repeat_interleave(group, 1)
    assert torch.equal(back.isnan(), wide)
    assert torch.equal(back[~wide], qb.int4_dequantize(clean)[~wide])
    x = rand(3, k, seed=1)
    h, h0 = qb.int4_linear_fwd(w, x), qb.int4_linear_fwd(clean, x)
    assert bool(h[:, 1:].isnan().all()) and torch.equal(h[:, 0], h0[:, 0])


def test_int4_beyond_32_bit_offsets():
    n, k = 2 ** 16 + 5, 65536  # codes of more than 2^31 bytes, more than 2^32 weights
    W = torch.zeros(n, k, dtype=BF, device=DEV)
    W[-7:] = rand(7, k, std=0.02, seed=1)
    w = qb.int4_quantize(W, group=128)
    q, s, z = ref.int4(W[-7:], 128, True)
    assert torch.equal(w.scale[-7:].cpu(), s) and torch.equal(w.zero_point[-7:].cpu().long(), torch.from_numpy(z))
    assert torch.equal(ref.int4_unpack(w.codes[-7:]).cpu().long(), torch.from_numpy(q))
    assert int(w.codes[:-7].count_nonzero()) == 0
    x = rand(2, k, seed=2)
    h = qb.int4_linear_fwd(w, x)
    part = qb.Int4Weight(7, k, 128, w.codes[-7:].clone(), w.scale[-7:].clone(), w.zero_point[-7:].clone())
    V = ref.int4_values(part.codes, part.scale, part.zero_point, 128)
    want, size = x.double() @ V.t(), x.double().abs() @ V.abs().t()
    # a group's sum is 8 accumulations (2^-22 of the sizes each at most), and the 512 groups of a row are joined by at most
    # 32 fp32 additions in a row per warp (64 groups over two at least) and 16 over the parts of k (2^-24 each): below 2^-17
    within(h[:, -7:], want, want.abs() * ref.HALF_STEP + size * 2.0 ** -17 + TINY)
    assert int(h[:, :-7].count_nonzero()) == 0
    back = qb.int4_dequantize(w, out=W)
    assert torch.equal(back[-7:], qb.int4_dequantize(part)) and int(back[:-7].count_nonzero()) == 0


# ---------------------------------------------------------------------------- SwiGLU

@pytest.mark.parametrize("scale", [1.0, 2.0 ** 40])
def test_swiglu_of_gates_far_below_zero(scale):
    # exp(-g) leaves fp32 on the way down: the results do not, by far, where up is large or g is above -104
    gate = torch.linspace(-103.0, -84.0, 64 * 32, device=DEV).to(BF).reshape(4, -1)
    up, dy = (rand(4, 512, seed=1).float() * scale).to(BF), rand(4, 512, seed=2)
    y, g8, u8 = qb.swiglu_act8_fwd(gate, up)
    # exp of a rounded argument and the products as in the other tests; below 2^-126 sigma is a multiple of 2^-149, and
    # exp, the quotient and two products may each be off by one
    def few(g, *factors):
        f = 1.0 + g.abs()
        for t in factors:
            f = f * (1.0 + t.abs())
        return f * 4.0 * 2.0 ** -149

    g, u = gate.double(), up.double()
    eta = (6.0 + 1.2 * g.abs()) * 2.0 ** -23
    want = ref.swiglu(g, u)
    assert float(want.abs().max()) > 2.0 ** -118 and int((want.abs() > 2.0 ** -126).sum()) > 500
    within(y, want, want.abs() * (ref.HALF_STEP + 1.01 * eta) + few(g, u) + TINY, "y")

    gg, gu, y8 = qb.swiglu_act8_bwd(g8, u8, dy)
    g, u, d = ref.act8_values(g8.codes, g8.absmax), ref.act8_values(u8.codes, u8.absmax), dy.double()
    eta = (8.0 + 1.2 * g.abs()) * 2.0 ** -23
    dg, du = ref.swiglu_grads(g, u, d)
    # 1 + g (1 - sigma) is near g here and does not cancel: two roundings
    within(gg, dg, dg.abs() * (ref.HALF_STEP + 1.01 * eta + 2.0 ** -22) + few(g, u, d) + TINY, "grad_gate")
    within(gu, du, du.abs() * (ref.HALF_STEP + 1.01 * eta) + few(g, d) + TINY, "grad_up")
    want = ref.swiglu(g, u)
    top = want.abs().reshape(4, -1, 64).amax(-1, keepdim=True).expand(-1, -1, 64).reshape(want.shape)
    rounding = top * (ref.HALF_STEP + 1.01 * eta) + few(g, u) + TINY
    within(ref.act8_values(y8.codes, y8.absmax), want, rounding + top * 1.02 / 254.0, "y8")


# ------------------------------------------------------------------- adapter gradients

@pytest.mark.parametrize("M,n,k,r", [(1100, 264, 320, 16), (1100, 264, 192, 64), (4100, 520, 64 * 21, 40)])
def test_grads_of_a_call_that_gives_its_waits_up_are_nan_and_the_next_call_runs(M, n, k, r):
    x8, gh, A, B = grad_inputs(M, n, k, r)
    drop = (0.1, 3, 1)
    want = qb.qlora_lora_grads_act8(x8, gh, A, B, 16.0, dropout=drop)
    for _ in range(2):
        ga, gb = qb.selftest_grads_give_up(x8, gh, A, B, 16.0, drop)
        torch.cuda.synchronize()
        assert bool(ga.isnan().all()) and torch.equal(gb, want[1])
        again = qb.qlora_lora_grads_act8(x8, gh, A, B, 16.0, dropout=drop)
        assert all(torch.equal(a, b) for a, b in zip(again, want))


# few tokens over wide layers: blocks of 16 columns of the rank; odd widths and ranks, and the last block with one column
WIDE = [(120, 28672, 8192, 64), (33, 20001, 11008, 61), (17, 28672, 28672, 33), (1, 40000, 36864, 16)]


def takes_blocks_of_16(M, n, k, r):
    return M < 128 and ((n + 255) // 256 + (k + 255) // 256) * ((r + 15) // 16) > 2 * SMS


@pytest.mark.parametrize("M,n,k,r", WIDE)
def test_grads_few_tokens_of_wide_layers(M, n, k, r):
    assert takes_blocks_of_16(M, n, k, r)
    check_grads(*grad_inputs(M, n, k, r, seed=M), 16.0)


@pytest.mark.parametrize("M,n,k,r", [(120, 28672, 8192, 64), (33, 20001, 11008, 61)])
def test_grads_few_tokens_of_wide_layers_dropout(oracle, M, n, k, r):
    assert takes_blocks_of_16(M, n, k, r)
    p, seed, offset = 0.1, 987654321, 2 ** 32 - 5
    keep = torch.from_numpy(oracle.dropout_keep(seed, offset, p, M, k)).to(DEV)
    check_grads(*grad_inputs(M, n, k, r), 16.0, keep=keep.double(), dropout=(p, seed, offset))


@pytest.mark.parametrize("M,n,k,r", [(1100, 264, 320, 48), (1100, 264, 320, 64), (1037, 201, 448, 64), (1200, 328, 192, 100),
                                     (1090, 203, 320, 129), (1152, 64, 2048, 32), (1300, 4096, 2048, 64)])
def test_grads_long_batch_dropout_ranks(oracle, M, n, k, r):
    p, seed, offset = 0.1, 1234567890123, 7
    keep = torch.from_numpy(oracle.dropout_keep(seed, offset, p, M, k)).to(DEV)
    check_grads(*grad_inputs(M, n, k, r, seed=r), 16.0, keep=keep.double(), dropout=(p, seed, offset))


@pytest.mark.parametrize("drop", [False, True])
def test_grads_long_batch_in_two_launches_of_the_second_kernel(oracle, drop):
    M, n, k, r = 1030, 36864, 2048, 64  # 144 + 16 column tiles: 148 in the first launch, 12 of the codes in the second
    p, seed, offset = 0.1, 5, 11
    args = grad_inputs(M, n, k, r, seed=1)
    keep = torch.from_numpy(oracle.dropout_keep(seed, offset, p, M, k)).to(DEV).double() if drop else None
    qb.launch_count(reset=True)
    check_grads(*args, 16.0, keep=keep, dropout=(p, seed, offset) if drop else None)
    assert SMS != 148 or qb.launch_count() == 3


def test_grads_beyond_32_bit_offsets_few_tokens():
    # grad_h of more than 2^31 values in rows of 17 million: all of them zero but the last columns
    M, n, k, r, last = 127, 17_000_001, 128, 4, 700
    x8 = qb.act8_quantize(rand(M, k, seed=1))
    gh = torch.zeros(M, n, dtype=BF, device=DEV)
    gh[:, -last:] = rand(M, last, seed=2)
    A, B = rand(r, k, std=0.01, seed=3), rand(n, r, std=0.01, seed=4)
    ga, gb = qb.qlora_lora_grads_act8(x8, gh, A, B, 8.0)
    x, s = ref.act8_values(x8.codes, x8.absmax), 2.0
    wa, wb, sa, sb = ref.lora_grads(x, gh[:, -last:].double(), A.double(), B[-last:].double(), s)
    # 2^-23 for each fp32 operation on the way, as check_grads counts them: the zeros add none
    unit = lambda features: ((5 * features / 64 + 8) + (3 * (M / 16 + 1) + 10) + 5) * 2.0 ** -23  # noqa: E731
    within(ga, wa, sa * unit(last) + 1e-30, "grad_A")
    within(gb[-last:], wb, sb * unit(k) + 1e-30, "grad_B")
    assert int(gb[:-last].count_nonzero()) == 0


def test_grads_beyond_32_bit_offsets_long_batch():
    # codes and grad_h of more than 2^31 values each: all zero but those of the last tokens
    M, n, k, r, last = 75_001, 28680, 28672, 16, 300
    x = torch.zeros(M, k, dtype=BF, device=DEV)
    x[-last:] = rand(last, k, seed=1)
    x8 = qb.act8_quantize(x)
    del x
    gh = torch.zeros(M, n, dtype=BF, device=DEV)
    gh[-last:] = rand(last, n, seed=2)
    A, B = rand(r, k, std=0.01, seed=3), rand(n, r, std=0.01, seed=4)
    ga, gb = qb.qlora_lora_grads_act8(x8, gh, A, B, 32.0)
    wa, wb, sa, sb = ref.lora_grads(ref.act8_values(x8.codes[-last:], x8.absmax[-last:]), gh[-last:].double(), A.double(),
                                    B.double(), 2.0)
    unit = lambda features: ((5 * features / 64 + 8) + (3 * (last / 16 + 1) + 10) + 5) * 2.0 ** -23  # noqa: E731
    within(ga, wa, sa * unit(n) + 1e-30, "grad_A")
    within(gb, wb, sb * unit(k) + 1e-30, "grad_B")


# ------------------------------------------------------------------- marshalling

def test_calls_without_the_compiled_marshalling_give_the_same(monkeypatch):
    x, up, dy, W = rand(6, 320, seed=1), rand(6, 320, seed=2), rand(6, 320, seed=3), rand(24, 320, std=0.02, seed=4)
    A, B = rand(8, 320, seed=5), rand(320, 8, seed=6)

    def step():
        a = qb.act8_quantize(x)
        y, g8, u8 = qb.swiglu_act8_fwd(x, up)
        gg, gu, y8 = qb.swiglu_act8_bwd(g8, u8, dy)
        w = qb.int4_quantize(W, group=64)
        return (a.codes, a.absmax, qb.act8_dequantize(a), y, g8.codes, u8.absmax, gg, gu, y8.codes, w.codes, w.scale,
                w.zero_point, qb.int4_dequantize(w), qb.int4_linear_fwd(w, x), *qb.qlora_lora_grads_act8(a, up, A, B, 8.0))

    want = step()
    monkeypatch.setattr(qb, "_marshal", qb._NoMarshal())
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
