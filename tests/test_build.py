"""The build's host logic (no compiler run: the commands are recorded, and their outputs written by the test)."""
import importlib.util
import os
import subprocess

import pytest

from int8_quant_b200 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty package folder, and compilers that write a line into the file they are asked for."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "binding.cpp").write_text("")
    for k, v in {"HERE": tmp_path, "CSRC": csrc, "LIB": tmp_path / "libssd.so", "BINDING": tmp_path / "_binding.so",
                 "STAMP": tmp_path / "_binding.torch"}.items():
        monkeypatch.setattr(b, k, str(v), raising=False)

    class Tree:
        here, fail, runs = tmp_path, None, 0

        def text(self, name):
            p = tmp_path / name
            return p.read_text() if p.exists() else None

    t = Tree()

    def run(cmd, check, cwd):
        out = cmd[cmd.index("-o") + 1]
        if t.fail and any(a.endswith(t.fail) for a in cmd):
            raise subprocess.CalledProcessError(1, cmd)
        t.runs += 1
        with open(out, "w") as f:
            f.write(f"run {t.runs}")

    monkeypatch.setattr(subprocess, "run", run)
    return t


def test_a_binding_that_fails_leaves_the_library_as_it_was(tree):
    b.build()
    assert (tree.text("libssd.so"), tree.text("_binding.so")) == ("run 1", "run 2")
    tree.fail = "binding.cpp"
    with pytest.raises(subprocess.CalledProcessError):
        b.build(force=True)
    assert (tree.text("libssd.so"), tree.text("_binding.so")) == ("run 1", "run 2")
    assert sorted(os.listdir(tree.here)) == ["_binding.so", "_binding.torch", "csrc", "libssd.so"]


def test_without_torch_the_library_is_built_alone(tree, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    assert b.needs_build()
    b.build()
    assert tree.text("libssd.so") == "run 1" and tree.text("_binding.so") is None
    assert not b.needs_build()


def test_another_torch_needs_another_binding(tree, monkeypatch):
    import torch
    b.build()
    assert not b.needs_build()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert b.needs_build()
    b.build()
    assert tree.text("libssd.so") == "run 3" and tree.text("_binding.so") == "run 4" and not b.needs_build()


def test_a_binding_for_another_torch_is_not_used(monkeypatch):
    import torch
    from int8_quant_b200 import ssd
    assert ssd._binding().torch_version == torch.__version__
    monkeypatch.setattr(ssd, "_BINDING", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ImportError, match="0.0.1"):
        ssd._binding()


def test_a_binding_of_an_older_build_is_not_used(monkeypatch):
    from int8_quant_b200 import ssd
    monkeypatch.delattr(ssd._binding(), "torch_version")
    monkeypatch.setattr(ssd, "_BINDING", None)
    with pytest.raises(ImportError, match="older build"):
        ssd._binding()
