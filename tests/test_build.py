"""What build() compiles and links, with the compilers replaced by a recorder."""
import os
import subprocess
import sys

import pytest

from fp8_block_scaled_dynamic_gb300 import build as b


class Compilers:
    """Stands for nvcc and g++: notes each command's tool and output, and writes
    the output unless the tool is to fail."""

    def __init__(self):
        self.made, self.failing = [], set()

    def run(self, cmd, **kw):
        tool, out = os.path.basename(cmd[0]), cmd[cmd.index("-o") + 1]
        ok = tool not in self.failing
        if ok:
            with open(out, "w") as f:
                f.write(" ".join(cmd))
        self.made.append((tool, os.path.basename(out).split(".tmp")[0]))
        return subprocess.CompletedProcess(cmd, 0 if ok else 1, "", "" if ok else "no")

    def tools(self):
        t = sorted({tool for tool, _ in self.made})
        self.made.clear()
        return t


@pytest.fixture
def tree(tmp_path, monkeypatch):
    c = Compilers()
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmxgemm.so"))
    monkeypatch.setattr(b, "BIND", str(tmp_path / "_attn_bind.so"))
    monkeypatch.setattr(b.subprocess, "run", c.run)
    monkeypatch.setattr(b, "nvcc", lambda: "nvcc")
    return c


def test_everything_once_then_nothing(tree):
    b.build()
    assert {out for _, out in tree.made} == {s.replace(".cu", ".o") for s in b.SOURCES} | {
        "libmxgemm.so", "bind.o", "_attn_bind.so"}
    tree.made.clear()
    b.build()
    assert tree.made == []
    b.build(force=True)
    assert tree.tools() == ["g++", "nvcc"]


def test_the_library_needs_no_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.BIND) and tree.tools() == ["nvcc"]
    monkeypatch.undo()


def test_a_module_that_does_not_compile_leaves_the_library(tree):
    tree.failing.add("g++")
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BIND)
    tree.failing.clear()
    tree.made.clear()
    b.build()
    assert os.path.exists(b.BIND) and tree.tools() == ["g++"]


@pytest.mark.parametrize("what", ["torch", "Python"])
def test_a_module_for_another_torch_or_python_is_built_anew(tree, monkeypatch, what):
    import torch
    b.build()
    tree.made.clear()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.1")
    else:
        monkeypatch.setattr(sys, "version", "9.9 (another)")
    b.build()
    assert tree.tools() == ["g++"]
    b.build()
    assert tree.made == []
