"""The optional module of csrc/torch: it is built only where torch has all that it links to."""
import importlib.machinery
import importlib.util
import os
import types

import pytest

from paged_kv_cache_243_gb300 import _build


@pytest.fixture
def torch_tree(tmp_path, monkeypatch):
    """What a CUDA torch installs of headers and libraries, by name."""
    home = tmp_path / "torch"
    files = ["include/torch/csrc/autograd/python_variable.h", "include/c10/cuda/CUDAStream.h"] + \
        [f"lib/lib{n}.so" for n in ("torch_python", "torch", "torch_cuda", "torch_cpu", "c10_cuda", "c10")]
    for f in files:
        (home / f).parent.mkdir(parents=True, exist_ok=True)
        (home / f).touch()
    cuda = tmp_path / "cuda"
    (cuda / "include").mkdir(parents=True)
    (cuda / "include" / "cuda_runtime_api.h").touch()
    python = tmp_path / "python"
    python.mkdir()
    (python / "Python.h").touch()
    spec = importlib.machinery.ModuleSpec("torch", None, is_package=True)
    spec.submodule_search_locations.append(str(home))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else None)
    monkeypatch.setattr(_build, "sysconfig", types.SimpleNamespace(get_paths=lambda: {"include": str(python)},
                                                                   get_config_var=lambda name: "cpython-312"))
    monkeypatch.setattr(_build.shutil, "which", lambda name: "/usr/bin/" + name)
    return home, str(cuda)


def test_everything_there(torch_tree):
    home, cuda = torch_tree
    assert "-ltorch_cuda" in _build._torch_job(cuda)


@pytest.mark.parametrize("gone", ["lib/libtorch_cuda.so", "lib/libc10_cuda.so", "include/c10/cuda/CUDAStream.h"])
def test_a_torch_without_cuda_is_no_torch(torch_tree, gone):
    home, cuda = torch_tree
    os.unlink(home / gone)
    assert _build._torch_job(cuda) is None
