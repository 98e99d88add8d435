"""Which of the two libraries is compiled when, with compilers that only write
down that they were called."""

import os
import time
import types
import warnings

import pytest

from flashattention_backward_gb300 import _build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A tree of empty sources, and compilers that write empty outputs; fails: tools that find an error."""
    pkg = tmp_path / "pkg"
    csrc = pkg / "csrc"
    csrc.mkdir(parents=True)
    (tmp_path / "include").mkdir()
    t = types.SimpleNamespace(calls=[], fails=set(), csrc=csrc, header=tmp_path / "include" / "fa.h",
                              lib=pkg / "_lib" / "libfa.so", version="torch-a")
    for name in _build.SOURCES + [_build.TORCH_SOURCE, "a.cuh", "b.h"]:
        (csrc / name).write_text("")
    t.header.write_text("")
    t.binding = lambda: pkg / "_lib" / f"binding-{t.version}.so"

    def run(cmd, **kw):
        tool = "nvcc" if "nvcc" in os.path.basename(cmd[0]) else "cxx"
        if tool in t.fails:
            return types.SimpleNamespace(returncode=1, stdout="", stderr=f"{tool} found an error")
        t.calls.append(tool)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    for name, value in dict(PKG=str(pkg), CSRC=str(csrc), OUT_DIR=str(pkg / "_lib"), LIB=str(t.lib),
                            HEADER=str(t.header), torch_binding_path=lambda: str(t.binding()),
                            nvcc_path=lambda: "/bin/nvcc").items():
        monkeypatch.setattr(_build, name, value, raising=False)
    monkeypatch.setattr(_build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.delenv("CXX", raising=False)

    def build(**kw):
        t.calls.clear()
        with warnings.catch_warnings(record=True) as said:
            warnings.simplefilter("always")
            assert _build.build(**kw) == str(t.lib)
        return [str(w.message) for w in said]

    t.build = build
    return t


ALL = ["nvcc"] * (len(_build.SOURCES) + 1)


def touch(tree, path):
    """path is the only source that is newer than what was built."""
    now = time.time()
    for p in [tree.header, *tree.csrc.iterdir()]:
        os.utime(p, (now - 100, now - 100))
    for p in (tree.lib, tree.binding()):
        os.utime(p, (now - 50, now - 50))
    os.utime(path, (now - 10, now - 10))


def test_both_are_built_once(tree):
    assert tree.build() == [] and sorted(tree.calls) == ["cxx"] + ALL
    assert tree.lib.exists() and tree.binding().exists()
    assert tree.build() == [] and tree.calls == []
    assert tree.build(force=True) == [] and sorted(tree.calls) == ["cxx"] + ALL


def test_the_library_needs_no_binding(tree):
    """A binding that does not compile is reported by itself; the library is there."""
    tree.fails = {"cxx"}
    said = tree.build()
    assert tree.calls == ALL and tree.lib.exists() and not tree.binding().exists()
    assert len(said) == 1 and "cxx found an error" in said[0]
    assert len(tree.build()) == 1 and tree.calls == []
    tree.fails = set()
    assert tree.build() == [] and tree.calls == ["cxx"]


def test_a_library_that_does_not_compile_is_an_error(tree):
    tree.fails = {"nvcc"}
    with pytest.raises(RuntimeError, match="nvcc found an error"):
        _build.build()


def test_another_pytorch_compiles_the_binding_alone(tree):
    tree.build()
    tree.version = "torch-b"
    assert tree.build() == [] and tree.calls == ["cxx"]


def test_each_follows_its_own_sources(tree):
    tree.build()
    touch(tree, tree.csrc / _build.TORCH_SOURCE)
    tree.build()
    assert tree.calls == ["cxx"]
    touch(tree, tree.csrc / "a.cuh")
    tree.build()
    assert tree.calls == ALL
    touch(tree, tree.header)
    tree.build()
    assert sorted(tree.calls) == ["cxx"] + ALL


def test_a_stale_binding_is_not_left_behind(tree):
    tree.build()
    touch(tree, tree.csrc / _build.TORCH_SOURCE)
    tree.fails = {"cxx"}
    assert len(tree.build()) == 1
    assert tree.lib.exists() and not tree.binding().exists()
