"""Build libpkv.so in-tree with nvcc for sm_103a (no torch extension machinery).

Each translation unit compiles in parallel; the shared library is relinked only
when a source or header is newer than it. Beside it, where torch is installed with its headers
and CUDA libraries: torch_library(), host code that makes some calls from torch tensors without Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libpkv.so")
TORCH_SRC = os.path.join(CSRC, "torch", "torch_calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def torch_library(version: str) -> str:
    """Where the module for this torch and this Python is: it has the layouts of both compiled in."""
    return os.path.join(OUT_DIR, f"_pkv_torch.{version}.{sysconfig.get_config_var('SOABI')}.so")


_TORCH_LINKS = ("torch_python", "torch", "torch_cuda", "torch_cpu", "c10_cuda", "c10")


def _torch_job(cuda: str):
    """(the command that builds the module for the torch that is installed, with ".tmp" behind its name; that name). None
    where torch, its headers or its CUDA libraries are not there."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    home, python = spec.submodule_search_locations[0], sysconfig.get_paths()["include"]
    include, libs = os.path.join(home, "include"), os.path.join(home, "lib")
    needed = [os.path.join(python, "Python.h"), os.path.join(include, "torch", "csrc", "autograd", "python_variable.h"),
              os.path.join(include, "c10", "cuda", "CUDAStream.h"), os.path.join(cuda, "include", "cuda_runtime_api.h"),
              os.path.join(home, "version.py")] + [os.path.join(libs, f"lib{n}.so") for n in _TORCH_LINKS]
    if not (all(map(os.path.exists, needed)) and shutil.which("g++")):
        return None
    with open(os.path.join(home, "version.py")) as f:
        version = re.search(r"^__version__ = ['\"]([^'\"]+)['\"]", f.read(), re.M)
    if not version:
        return None
    paths = [INCLUDE, include, os.path.join(include, "torch", "csrc", "api", "include"), python, os.path.join(cuda, "include")]
    target = torch_library(version.group(1))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared"] + [x for p in paths for x in ("-I", p)] + \
        [TORCH_SRC, "-o", target + ".tmp", "-L", libs] + ["-l" + n for n in _TORCH_LINKS], target


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile every source under csrc/ and link _lib/libpkv.so; return its path."""
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    headers = _headers()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            if src.endswith(".cu"):
                cmd = [nvcc] + ARCH + ["-lineinfo"] + common + ["-c", src, "-o", obj]
            else:
                cmd = [nvcc] + common + ["-c", src, "-o", obj]
            jobs.append(cmd)

    tool_jobs = len(jobs)
    torch_cmd, torch_lib = _torch_job(os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))) or (None, None)
    if torch_cmd and (force or _stale(torch_lib, [TORCH_SRC] + headers)):
        jobs.append(torch_cmd)
    else:
        torch_cmd = None

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    if jobs:
        workers = max(1, min(len(jobs), os.cpu_count() or 4))
        with cf.ThreadPoolExecutor(workers) as ex:
            for cmd, r in ex.map(run, jobs):
                if verbose or r.returncode != 0:
                    sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
                if r.returncode != 0:
                    raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd[-3:])}")
    if torch_cmd:
        os.replace(torch_lib + ".tmp", torch_lib)
    if force or tool_jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("linking libpkv.so failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
