"""Build libemb.so (the CUDA library behind include/emb.h) in-tree for sm_103a.

Each .cu file under csrc/ is compiled to an object in parallel, then linked into a shared
library next to this file.  The CUDA runtime is linked statically, so the library loads
on a machine without a GPU (it only needs the driver when a call reaches the device).  The
Python side of the expert tower's calls (csrc/py_tower.cpp, against torch's headers) becomes
_tower.so beside it, linked to the library; the library itself needs no torch, and where there is
none it is all that is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libemb.so")
TOWER_SRC = os.path.join(CSRC, "py_tower.cpp")
TOWER_OBJ = os.path.join(BUILD, "py_tower.o")
TOWER = os.path.join(HERE, "_tower.so")  # (TOWER_OBJ's stamp: what it was compiled for)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libemb.so")
    return cand


def _flags(verbose: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def gxx() -> str:
    return shutil.which("g++") or "g++"


def torch_root():
    """Where torch is installed (found without importing it); None: nowhere."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def torch_dirs(what: str):
    """torch's include or lib directories."""
    root = torch_root()
    if what == "lib":
        return [os.path.join(root, "lib")]
    inc = os.path.join(root, "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include")]


def torch_version() -> str:
    """torch's version as it says it itself (read without importing it)."""
    import re
    path = os.path.join(torch_root(), "version.py")
    with open(path) as f:
        found = re.search(r"^__version__\s*=\s*['\"]([^'\"]*)['\"]", f.read(), re.M)
    if not found:
        raise RuntimeError(f"{path} gives no version")
    return found.group(1)


def _tower_flags():
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    dirs = torch_dirs("include") + [cuda, sysconfig.get_paths()["include"]]
    return ["-O2", "-std=c++17", "-fPIC", f'-DEMB_TORCH_VERSION="{torch_version()}"',
            "-I" + os.path.join(ROOT, "include")] + [f"-isystem{d}" for d in dirs]


def _tower_stamp() -> str:
    """What _tower.so depends on beside the sources: it reads torch's and Python's objects in place,
    so it serves the versions that it was compiled for and no other."""
    return "\n".join([str(sysconfig.get_config_var("SOABI")), gxx()] + _tower_flags() + torch_dirs("lib")) + "\n"


def _stamped(stamp: str) -> bool:
    try:
        with open(TOWER_OBJ + ".stamp") as f:
            return f.read() == stamp
    except OSError:
        return False


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "emb.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, jobs: int = 0) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [(s, o) for s, o in zip(srcs, objs) if force or _stale(o, s)]
    tower = torch_root() is not None
    stamp = _tower_stamp() if tower else ""
    tower_todo = tower and (force or _stale(TOWER_OBJ, TOWER_SRC) or not _stamped(stamp))
    nv = nvcc()

    def compile_one(s, o):
        tmp = o + f".tmp{os.getpid()}"
        cmd = ([nv] + _flags(verbose) if s != TOWER_SRC else [gxx()] + _tower_flags()) + ["-c", s, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiler failed on {os.path.basename(s)}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, o)
        return r.stderr

    with cf.ThreadPoolExecutor(max_workers=jobs or max(1, min(len(todo) + 1, os.cpu_count() or 4))) as ex:
        tower_job = ex.submit(compile_one, TOWER_SRC, TOWER_OBJ) if tower_todo else None
        logs = list(ex.map(compile_one, *zip(*todo))) if todo else []
    if todo or force or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nv] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of libemb.so failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if not tower:
        sys.stderr.write("torch is not installed: _tower.so (the Python side of the tower's calls) is not built\n")
    elif todo or tower_todo or not os.path.exists(TOWER):  # relinked to the new library
        if tower_job:
            logs.append(tower_job.result())
        tmp = TOWER + f".tmp{os.getpid()}"
        cmd = [gxx(), "-shared", TOWER_OBJ, "-o", tmp, "-L" + HERE, "-l:libemb.so", "-Wl,-rpath,$ORIGIN"]
        for d in torch_dirs("lib"):
            cmd += ["-L" + d, "-Wl,-rpath," + d]
        cmd += ["-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of _tower.so failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, TOWER)
        with open(TOWER_OBJ + ".stamp", "w") as f:
            f.write(stamp)
    if verbose:
        for l in logs:
            sys.stderr.write(l)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
