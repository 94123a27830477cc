"""Host-side checks of the 8-bit activation entry points beside those of test_lowbit_host.py (the addresses here are never
read: no call reaches a GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def qb():
    from bit_nf4_quantized_25_b200 import binding, build
    build.build()
    binding.load()
    return binding


P = ctypes.c_void_p
EINVAL, ESHAPE, EALIGN, EWORKSPACE = 1, 2, 3, 5


def test_the_give_up_self_test_refuses_what_it_does_not_take(qb):
    lib, r = qb.load(), ctypes.byref
    f = lib.qn_selftest_grads_give_up
    gh, A, B, ga, gb, ws = (P(0x40000000 + 0x10000000 * i) for i in range(6))
    x, d = qb.CAct8(1100, 128, 0x10000000, 0x20000000), qb.CDropout(0.1, 1, 0)
    size = qb.lora_grads_act8_workspace_size(1100, 96, 16)

    def call(x=x, d=d, gh=gh, rank=16, size=size):
        return f(None if x is None else r(x), gh, 96, A, B, rank, 32.0, None if d is None else r(d), ga, gb, ws, size, None)

    before = lib.qn_launch_count(0)
    assert call(x=None) == EINVAL
    assert call(x=qb.CAct8(1024, 128, 0x10000000, 0x20000000)) == ESHAPE  # those take kernels without such waits
    assert call(d=None) == EINVAL and call(d=qb.CDropout(0.0, 1, 0)) == EINVAL and call(d=qb.CDropout(1.0, 1, 0)) == EINVAL
    assert call(gh=None) == EINVAL and call(gh=P(0x40000002)) == EALIGN
    assert call(rank=0) == EINVAL and call(size=size - 1) == EWORKSPACE
    assert lib.qn_launch_count(0) == before


def test_the_package_offers_the_size_of_every_workspace_that_a_call_takes(qb):
    import inspect

    import bit_nf4_quantized_25_b200 as package
    takes = {name for name in package.__all__ if "workspace" in inspect.signature(getattr(package, name)).parameters}
    assert takes == {"nf4_quantize", "qlora_linear_fwd", "qlora_linear_bwd_x", "qlora_lora_grads", "qlora_lora_grads_act8"}
    assert package.quantize_workspace_size(64, 128) > 0 and package.linear_workspace_size(3, 64, 128, 8) > 0
    assert package.lora_grads_workspace_size(40, 8) > 0
    assert package.lora_grads_act8_workspace_size(1100, 97, 8) > package.lora_grads_act8_workspace_size(1100, 96, 8) > 0
    assert set(package.__all__) <= set(dir(package)) and len(package.__all__) == len(set(package.__all__))
