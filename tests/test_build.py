"""The build's order: the C library needs nvcc alone and is there whatever becomes of the binding."""

import os
import subprocess

import pytest

from tiled_attention_fa_gb300 import build


@pytest.mark.parametrize("how", ["compile", "headers"])
def test_the_library_is_linked_without_the_binding(tmp_path, monkeypatch, how):
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "_compile", lambda unit, verbose: (unit, str(tmp_path / unit), 0, ""))

    (tmp_path / "binding.so").write_text("of an earlier build")

    def run(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", run)

    def binding():
        if how == "headers":
            raise ImportError("no torch")
        return "binding.cpp", str(tmp_path / "b.o"), 1, "Python.h: no such file"
    monkeypatch.setattr(build, "_compile_binding", binding)
    with pytest.raises(RuntimeError, match="binding"):
        build.build(quiet=True)
    assert os.path.exists(tmp_path / "lib.so") and not os.path.exists(tmp_path / "binding.so")
