"""The 8-bit activations and the 4-bit integer weights on the GPU where their other tests do not reach: weights that are not
finite, gates far below zero, waits that run out, calls without the compiled
marshalling. Compared with 64-bit forms (lowbit_ref)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import lowbit_ref as ref
from bit_nf4_quantized_25_b200 import binding as qb
from test_lowbit_gpu import BF, DEV, TINY, grad_inputs, rand, within


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
