"""What the build makes anew: the binding's helpers are compiled against the installed torch and Python."""
import os

import pytest

from serve_invariant_moe_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of its own, where compiling and linking write empty files; the list of what was compiled."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (tmp_path / "include").mkdir()
    for name in ("a.cu", "marshal.cpp"):
        (csrc / name).write_text("")
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "marshal.so"))
    compiled = []

    def compile_(src, verbose_ptxas=False):
        compiled.append(os.path.basename(src))
        open(build._object(src), "w").close()
        return build._object(src), ""

    monkeypatch.setattr(build, "_compile", compile_)
    monkeypatch.setattr(build, "_link", lambda cmd: open(cmd[cmd.index("-o") + 1], "w").close())
    return compiled


def test_another_torch_or_python_compiles_the_helpers_again(tree, monkeypatch):
    import sys

    import torch
    build.build()
    assert sorted(tree) == ["a.cu", "marshal.cpp"]
    tree.clear()
    build.build()
    assert tree == []
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    build.build()
    assert tree == ["marshal.cpp"]
    tree.clear()
    build.build()
    assert tree == []
    monkeypatch.setattr(sys, "version", "0 " + sys.version)
    build.build()
    assert tree == ["marshal.cpp"]
