"""The build script's own logic, with the compilers replaced: what is built, in which order, and when."""
import os
import subprocess
import types

import pytest
import torch

from bit_nf4_quantized_25_b200 import build as b


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Commands are recorded and write their output file; those whose program is in `broken` fail."""
    state = types.SimpleNamespace(ran=[], broken=set())

    def run(cmd, **kw):
        program = os.path.basename(cmd[0])
        state.ran.append(program)
        if program in state.broken:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such thing")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(b, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(b, "PKG", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_marshal.so"), raising=False)
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "obj"))
    return state


def test_the_library_is_built_where_the_extension_module_cannot_be(compilers):
    compilers.broken.add("g++")
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert os.path.exists(b.LIB)
    assert compilers.ran[-1] == "g++" and compilers.ran.count("nvcc") == len(b._sources()) + 1
    compilers.broken.clear()
    compilers.ran.clear()
    assert b.build() == b.LIB and compilers.ran == ["g++"]  # the library is up to date


def test_the_extension_module_is_built_anew_for_another_torch(compilers, monkeypatch):
    first = b.build_marshal()
    assert b.build_marshal() == first and compilers.ran == ["g++"]
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    second = b.build_marshal()
    assert second != first and os.path.exists(second) and compilers.ran == ["g++"] * 2


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    from bit_nf4_quantized_25_b200 import binding as qb
    b.build()
    monkeypatch.setattr(qb, "_marshal", None)
    assert qb._native().__file__ == b.marshal_path()
    names = {os.path.basename(b.marshal_path())}
    for attribute, value in (("__version__", "0.0.1"), ("compiled_with_cxx11_abi", lambda: not torch._C._GLIBCXX_USE_CXX11_ABI)):
        with monkeypatch.context() as m:
            m.setattr(torch, attribute, value)
            names.add(os.path.basename(b.marshal_path()))
            m.setattr(qb, "_marshal", None)
            with pytest.warns(RuntimeWarning, match="missing"):
                assert isinstance(qb._native(), qb._NoMarshal)
    assert len(names) == 3


def test_calls_take_the_general_way_without_the_extension_module(monkeypatch, tmp_path):
    from bit_nf4_quantized_25_b200 import binding as qb
    b.build()
    monkeypatch.setattr(qb, "_marshal", None)
    monkeypatch.setattr(b, "PKG", str(tmp_path))
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="bit_nf4_quantized_25_b200.build"), \
            pytest.raises(ValueError, match="not on a CUDA device"):  # the general way's answer
        qb.act8_quantize(x)
