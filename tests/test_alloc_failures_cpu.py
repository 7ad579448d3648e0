"""Host memory that runs out inside an allocator call: the call is refused and nothing has changed."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_call_without_memory_changes_nothing(tmp_path):
    exe = str(tmp_path / "alloc_failures")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "paged_kv_cache_243_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "alloc_failures.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[-1]) > 10
