"""What the build makes, and when, with compilers that only write their outputs (CPU only)."""
import os
import subprocess
import types

import pytest

from block_sparse_top_msa_gb300 import buildlib


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs in a folder of their own; `tree.ran` lists the compilers called, `tree.broken` those that fail."""
    t = types.SimpleNamespace(ran=[], broken=set())
    for name, to in (("HERE", tmp_path), ("OBJ", tmp_path / "_build"), ("LIB", tmp_path / "libmsa.so"), ("BINDING", tmp_path / "_binding.so"),
                     ("STAMP", tmp_path / "_build" / "binding.stamp")):
        monkeypatch.setattr(buildlib, name, str(to), raising=name != "STAMP")

    def run(cmd, **kw):
        tool = os.path.basename(cmd[0])
        t.ran.append(tool)
        if tool in t.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(buildlib.subprocess, "run", run)
    return t


def test_both_are_built_once(tree):
    assert buildlib.build() == buildlib.LIB
    assert os.path.exists(buildlib.LIB) and os.path.exists(buildlib.BINDING)
    assert tree.ran.count("g++") == 2 and tree.ran.count("nvcc") == len(buildlib.sources()) + 1
    tree.ran.clear()
    buildlib.build()
    assert tree.ran == [] and buildlib.up_to_date()


def test_the_library_is_built_where_the_binding_cannot_be(tree):
    """The calls that go through ctypes need neither g++ nor torch's headers."""
    tree.broken.add("g++")
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert buildlib.build() == buildlib.LIB
    assert os.path.exists(buildlib.LIB) and not os.path.exists(buildlib.BINDING) and not buildlib.up_to_date()
    tree.ran.clear()
    tree.broken.clear()
    buildlib.build()  # the library stays, the binding is made up for
    assert tree.ran == ["g++", "g++"] and buildlib.up_to_date()


def test_a_library_that_does_not_compile_is_an_error(tree):
    tree.broken.add("nvcc")
    with pytest.raises(RuntimeError, match="nvcc"):
        buildlib.build()
    assert not os.path.exists(buildlib.LIB)


def test_another_torch_makes_the_binding_anew(tree, monkeypatch):
    import torch
    buildlib.build()
    tree.ran.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not buildlib.up_to_date()
    buildlib.build()
    assert tree.ran == ["g++", "g++"] and buildlib.up_to_date()
