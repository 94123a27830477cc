"""The build script's own logic, with the compilers replaced: what is built, in which order, and when."""
import os
import subprocess
import types

import pytest

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
