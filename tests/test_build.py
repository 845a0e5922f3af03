"""What the build makes where torch is missing or not what it was.  Compilers are stood in for; no GPU
is needed."""
import importlib.util
import os
import subprocess
import sys
import types

import pytest

from conftest import ROOT

PACKAGE = os.path.join(ROOT, "recommender_model_embedding_gb300")


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build script with its products in tmp_path and compilers that write empty files; `ran`: their
    commands, `fails`: a text in the command of the one that fails."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PACKAGE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.BUILD, b.LIB, b.TOWER = (str(tmp_path / n) for n in ("_build", "libemb.so", "_tower.so"))
    b.TOWER_OBJ = os.path.join(b.BUILD, "py_tower.o")
    b.ran, b.fails = [], None

    def run(cmd, **kw):
        b.ran.append(cmd)
        if b.fails and any(b.fails in c for c in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="refused")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    b.subprocess = types.SimpleNamespace(run=run)
    b.nvcc = lambda: "/usr/local/cuda/bin/nvcc"
    return b


def _no_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_is_built_without_torch(build, monkeypatch):
    _no_torch(monkeypatch)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.TOWER) and not any("py_tower" in c for cmd in build.ran for c in cmd)


@pytest.mark.parametrize("fails", ["py_tower.cpp", "-ltorch_python"])
def test_library_is_there_when_the_tower_module_fails(build, fails):
    build.fails = fails
    with pytest.raises(RuntimeError, match="refused"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TOWER)


def test_second_build_has_nothing_to_do(build):
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.TOWER)
    build.ran.clear()
    build.build()
    assert not build.ran


def test_package_imports_without_the_tower_module():
    """Everything but the tower's calls works without _tower.so, and those say what is missing."""
    from helpers import build_lib
    build_lib()
    code = """
import os
there = os.path.exists
os.path.exists = lambda p: False if str(p).endswith("_tower.so") else there(p)
import recommender_model_embedding_gb300 as E
assert E.expert_sort_workspace(4, 2, 8) == 0
for call in (lambda: E.expert_dispatch(None, None, None), lambda: E.clip_grads([], 1.0, None)):
    try:
        call()
    except ImportError as e:
        assert "_tower.so is missing" in str(e)
    else:
        raise AssertionError("no ImportError")
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
