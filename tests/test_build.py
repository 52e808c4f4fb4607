"""What the in-tree build makes of what it finds, with compilers that only write their output."""
import os
import subprocess
import types

import pytest

torch = pytest.importorskip("torch")

from softmax_mx_block_gb300 import _build  # noqa: E402


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs in a folder of their own; the commands run, and those told to fail."""
    state = types.SimpleNamespace(ran=[], fails=())
    monkeypatch.setattr(_build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libfsa.so"))
    monkeypatch.setattr(_build, "TORCH_MODULE", str(tmp_path / "_fsa_torch.so"))

    def run(cmd, **kw):
        state.ran.append(cmd)
        if os.path.basename(cmd[0]) in state.fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build.subprocess, "run", run)
    return state


def compilers(state):
    return {os.path.basename(c[0]) for c in state.ran}


def test_both_are_built_once(tree):
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB) and os.path.exists(_build.TORCH_MODULE)
    assert compilers(tree) == {"nvcc", "g++"}
    tree.ran.clear()
    assert _build.build() == _build.LIB and tree.ran == []


def test_the_library_needs_no_torch_headers(tree, monkeypatch):
    """Neither a failing g++ nor a torch without headers keeps libfsa.so from being built."""
    tree.fails = ("g++",)
    with pytest.warns(RuntimeWarning, match="no header"):
        assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.TORCH_MODULE)

    def no_flags():
        raise ImportError("no torch here")

    monkeypatch.setattr(_build, "_torch_flags", no_flags)
    os.remove(_build.LIB)
    with pytest.warns(RuntimeWarning, match="no torch here"):
        assert _build.build(force=True) == _build.LIB
    assert os.path.exists(_build.LIB)
    tree.ran.clear()
    os.remove(_build.LIB)
    _build.build_library()
    assert compilers(tree) == {"nvcc"}
    with pytest.raises(ImportError, match="no torch here"):
        _build.build_torch_module()


def test_another_torch_rebuilds_the_module(tree, monkeypatch):
    _build.build()
    tree.ran.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    _build.build_torch_module()
    assert compilers(tree) == {"g++"}
    tree.ran.clear()
    _build.build_torch_module()
    assert tree.ran == []
