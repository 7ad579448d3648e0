"""The optional module of csrc/torch: it is built only where torch has all that it links to, belongs to one torch
and one Python, and loads for every cache or for none."""
import importlib.machinery
import importlib.util
import os
import threading
import time
import types

import pytest

from paged_kv_cache_243_gb300 import _build, binding


@pytest.fixture
def torch_tree(tmp_path, monkeypatch):
    """What a CUDA torch installs of headers and libraries, by name."""
    home = tmp_path / "torch"
    files = ["include/torch/csrc/autograd/python_variable.h", "include/c10/cuda/CUDAStream.h"] + \
        [f"lib/lib{n}.so" for n in ("torch_python", "torch", "torch_cuda", "torch_cpu", "c10_cuda", "c10")]
    for f in files:
        (home / f).parent.mkdir(parents=True, exist_ok=True)
        (home / f).touch()
    (home / "version.py").write_text("from typing import Optional\n__version__ = '9.8.7+cu130'\n")
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
    cmd, target = _build._torch_job(cuda)
    assert target == _build.torch_library("9.8.7+cu130") and target + ".tmp" in cmd and "-ltorch_cuda" in cmd


@pytest.mark.parametrize("gone", ["lib/libtorch_cuda.so", "lib/libc10_cuda.so", "include/c10/cuda/CUDAStream.h", "version.py"])
def test_a_torch_without_cuda_is_no_torch(torch_tree, gone):
    home, cuda = torch_tree
    os.unlink(home / gone)
    assert _build._torch_job(cuda) is None


def test_another_torch_or_python_has_another_module(monkeypatch):
    names = {_build.torch_library("2.9.1+cu130"), _build.torch_library("2.11.0+cu130")}
    monkeypatch.setattr(_build, "sysconfig", types.SimpleNamespace(get_config_var=lambda name: "cpython-399"))
    names.add(_build.torch_library("2.11.0+cu130"))
    assert len(names) == 3


def test_a_module_that_does_not_load_raises_every_time(tmp_path, monkeypatch):
    bad = tmp_path / "_pkv_torch.so"
    bad.write_bytes(b"no library")
    monkeypatch.setattr(binding, "_torch_calls", None)
    monkeypatch.setattr(_build, "torch_library", lambda version: str(bad))
    for _ in range(2):
        with pytest.raises(ImportError):
            binding.torch_calls()
    monkeypatch.setattr(_build, "torch_library", lambda version: str(tmp_path / "none.so"))
    assert binding.torch_calls() is None


def test_threads_during_the_load_get_the_module(tmp_path, monkeypatch):
    so = tmp_path / "_pkv_torch.so"
    so.touch()
    monkeypatch.setattr(binding, "_torch_calls", None)
    monkeypatch.setattr(_build, "torch_library", lambda version: str(so))
    monkeypatch.setattr(binding, "lib", lambda: types.SimpleNamespace(
        pkv_rotary_append=binding.ctypes.c_void_p(1), pkv_tree_attention=binding.ctypes.c_void_p(2),
        pkv_keep_tokens=binding.ctypes.c_void_p(3)))
    loads = []

    class Loader(importlib.machinery.SourceFileLoader):
        def exec_module(self, module):
            loads.append(module)
            time.sleep(0.2)
            module.bind = lambda *a: None

    monkeypatch.setattr(importlib.util, "spec_from_file_location",
                        lambda name, path: importlib.machinery.ModuleSpec(name, Loader(name, path)))
    got = []
    threads = [threading.Thread(target=lambda: got.append(binding.torch_calls())) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(loads) == 1 and got == [loads[0]] * 4
