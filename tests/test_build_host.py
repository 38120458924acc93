"""What a build does without: the C library is built and loaded without g++ and
torch's headers; the binding is built again for another torch.  The compilers are
stand-ins (no GPU needed)."""
import os
import subprocess
import types

import pytest
import torch

from bit_weight_delta_gb300 import _build


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Outputs under tmp_path; the commands that ran, by program name."""
    ran = []

    def run(cmd, **kw):
        name = os.path.basename(cmd[0])
        if name in run.missing:
            raise FileNotFoundError(cmd[0])
        ran.append(name)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    run.missing = set()
    monkeypatch.setattr(subprocess, "run", run)
    for name, value in (("BUILD_DIR", tmp_path / "objects"), ("LIB_PATH", tmp_path / "lib.so"),
                        ("BINDING_PATH", tmp_path / "binding.so"),
                        ("BINDING_STAMP", tmp_path / "objects" / "binding.txt")):
        monkeypatch.setattr(_build, name, str(value), raising=False)
    return types.SimpleNamespace(ran=ran, missing=run.missing)


def test_the_library_needs_no_cxx_compiler(compilers):
    compilers.missing.add("g++")
    assert os.path.exists(_build.build())
    assert set(compilers.ran) == {"nvcc"}
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        _build.build_binding()


def test_a_current_library_is_not_built_for_want_of_the_binding(compilers):
    _build.build()
    del compilers.ran[:]
    _build.build()
    assert compilers.ran == []
    _build.build_binding()
    assert compilers.ran == ["g++"]


def test_the_binding_is_built_once_and_again_for_another_torch(compilers, monkeypatch):
    for _ in range(2):
        _build.build_all()
    assert compilers.ran.count("g++") == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    _build.build_all()
    assert compilers.ran.count("g++") == 2 and compilers.ran.count("nvcc") == len(_build.SOURCES) + 1
