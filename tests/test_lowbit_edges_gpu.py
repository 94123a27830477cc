"""The 8-bit activations and the 4-bit integer weights on the GPU where their other tests do not reach: weights that are not
finite. Compared with 64-bit forms (lowbit_ref)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import lowbit_ref as ref
from bit_nf4_quantized_25_b200 import binding as qb
from test_lowbit_gpu import DEV, rand


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
