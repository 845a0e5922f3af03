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


def test_tower_module_is_built_again_for_another_torch(build, tmp_path, monkeypatch):
    """A new torch version, a torch elsewhere or another Python rebuild the module and nothing else."""
    def torch_at(name, version):
        root = tmp_path / name / "torch"
        root.mkdir(parents=True, exist_ok=True)
        (root / "__init__.py").touch()
        (root / "version.py").write_text(f"__all__ = ['__version__']\n__version__ = '{version}'\n")
        spec = types.SimpleNamespace(origin=str(root / "__init__.py"))
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: spec if n == "torch" else find(n, *a))

    def again():
        build.ran.clear()
        build.build()
        done = [sum(text in c for cmd in build.ran for c in cmd) for text in ("py_tower.cpp", "-ltorch_python")]
        assert len(build.ran) == sum(done)
        build_once_more = len(build.ran)
        build.build()
        assert len(build.ran) == build_once_more
        return done

    torch_at("a", "2.9.1")
    build.build()
    assert again() == [0, 0]
    torch_at("a", "2.11.0+cu130")
    assert again() == [1, 1]
    torch_at("b", "2.11.0+cu130")
    assert again() == [1, 1]
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-x")
    assert again() == [1, 1]
    # a module whose link failed is not taken for the new one
    torch_at("b", "2.12.0")
    build.fails = "-ltorch_python"
    with pytest.raises(RuntimeError):
        build.build()
    build.fails = None
    assert again() == [1, 1]


def test_tower_module_of_another_torch_is_refused():
    from helpers import build_lib
    build_lib()
    code = """
import torch
import recommender_model_embedding_gb300 as E
real, torch.__version__ = torch.__version__, "0.1"
for _ in range(2):
    try:
        E.expert_dispatch(None, None, None)
    except ImportError as e:
        assert "this is 0.1" in str(e), e
    else:
        raise AssertionError("no ImportError")
torch.__version__ = real
try:
    E.expert_dispatch(None, None, None)
except ValueError:
    pass
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


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
