"""The build script with compilers that only note that they were called: what is rebuilt when, and what without torch."""
import importlib.util
import os
import stat
import sys
import types

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_sparse_attention_head_b200")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the tree's shape with empty sources; called() names what was written since it was last asked."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PACKAGE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    here, log = tmp_path / "package", tmp_path / "log"
    (here / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    for f in [*b.SOURCES, "binding.cpp", "kv4.cuh"]:
        (here / "csrc" / f).touch()
    (tmp_path / "include" / "msa.h").touch()
    log.touch()
    compiler = tmp_path / "compiler"
    compiler.write_text(f'#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\ntouch "$2"\nbasename "$2" >> {log}\n')
    compiler.chmod(compiler.stat().st_mode | stat.S_IXUSR)
    for name, path in (("HERE", here), ("CSRC", here / "csrc"), ("LIB", here / "libmsa.so"), ("BINDING", here / "_binding.so"),
                       ("NVCC", compiler)):
        monkeypatch.setattr(b, name, str(path))
    monkeypatch.setattr(b, "CXX", str(compiler), raising=False)
    monkeypatch.setattr(b, "BINDING_FOR", str(here / "_binding.for"), raising=False)
    real = b.subprocess.check_call  # the host compiler under its own name
    monkeypatch.setattr(b.subprocess, "check_call", lambda c, **k: real([str(compiler), *c[1:]] if c[0] == "g++" else c, **k))

    def called():
        names = [x for x in log.read_text().split() if not x.endswith(".o")]
        log.write_text("")
        return names

    def newer(path):
        t = max(os.path.getmtime(os.path.join(d, f)) for d, _, fs in os.walk(tmp_path) for f in fs) + 10
        os.utime(path, (t, t))
        return t

    return types.SimpleNamespace(b=b, called=called, newer=newer, here=here, root=tmp_path)


def _settle(tree):
    """The outputs are newer than every source."""
    for f in ("libmsa.so", "_binding.so"):
        if (tree.here / f).exists():
            tree.newer(tree.here / f)


def _without_torch(monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n.split(".")[0] == "torch" else real(n, *a))
    for n in [m for m in sys.modules if m.split(".")[0] == "torch"]:
        monkeypatch.delitem(sys.modules, n)
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it raises ImportError


def test_the_library_is_built_without_torch(tree, monkeypatch):
    _without_torch(monkeypatch)
    assert tree.b.build() == tree.b.LIB
    assert tree.called() == ["libmsa.so"]
    _settle(tree)
    assert tree.b.build() == tree.b.LIB and tree.called() == []  # and is not stale for want of the binding


def test_the_binding_is_built_anew_for_another_torch_or_source(tree, monkeypatch):
    torch = pytest.importorskip("torch")
    tree.b.build()
    assert tree.called() == ["libmsa.so", "_binding.so"]
    _settle(tree)
    tree.b.build()
    assert tree.called() == []
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    tree.b.build()
    assert tree.called() == ["_binding.so"]
    tree.b.build()
    assert tree.called() == []
    tree.newer(tree.here / "csrc" / "binding.cpp")
    tree.b.build()
    assert tree.called() == ["_binding.so"]
    _settle(tree)
    tree.newer(tree.here / "csrc" / "kv4.cuh")
    tree.b.build()
    assert tree.called() == ["libmsa.so"]
    _settle(tree)
    tree.newer(tree.root / "include" / "msa.h")
    tree.b.build()
    assert tree.called() == ["libmsa.so", "_binding.so"]


def test_a_failed_binding_leaves_the_library_built(tree, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(tree.b, "CXX", "/bin/false", raising=False)
    import subprocess
    with pytest.raises(subprocess.CalledProcessError):
        tree.b.build()
    assert tree.called() == ["libmsa.so"]
    _settle(tree)
    with pytest.raises(subprocess.CalledProcessError):
        tree.b.build()
    assert tree.called() == []  # the binding alone is tried again
