"""The C library needs nvcc alone to build, and the package without its torch
module keeps every call but the operators that live there."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "allreduce_reduction_rank_gb300"


def copy(tmp_path, leave_out):
    """The package with its objects and their times, without some of what was built."""
    shutil.copytree(os.path.join(ROOT, PACKAGE), tmp_path / PACKAGE,
                    ignore=lambda d, names: [n for n in names if n in leave_out or n == "__pycache__"])
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    return tmp_path / PACKAGE / "_build"


@pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"), reason="no nvcc")
def test_the_library_builds_without_torch(tmp_path):
    out = copy(tmp_path, ("libsar.so", "_sar_torch.so"))
    # -S: no site-packages, so no torch; the objects are there and up to date
    run = subprocess.run([sys.executable, "-I", "-S", str(tmp_path / PACKAGE / "build.py")], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert (out / "libsar.so").exists() and not (out / "_sar_torch.so").exists()
    assert "torch" in run.stderr                        # it says what it left out


@pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"), reason="no nvcc")
def test_a_module_that_does_not_compile_leaves_the_library(tmp_path):
    out = copy(tmp_path, ("libsar.so", "_sar_torch.so"))
    (tmp_path / PACKAGE / "csrc" / "torch_binding.cpp").write_text("#error not today\n")
    run = subprocess.run([sys.executable, str(tmp_path / PACKAGE / "build.py")], capture_output=True, text=True)
    assert run.returncode != 0 and "not today" in run.stderr
    assert (out / "libsar.so").exists()


@pytest.mark.parametrize("broken", [False, True], ids=["missing", "built for another torch"])
def test_the_package_imports_without_its_torch_module(tmp_path, broken):
    out = copy(tmp_path, ("_sar_torch.so",))
    if broken:
        (out / "_sar_torch.so").write_bytes(b"not a library")
    code = ("import allreduce_reduction_rank_gb300 as sar\n"
            "assert sar.sar_rsag_chunk(1024, 4, 'fp16') > 0 and sar.sar_expert_rows(4, 2, 8) == 8\n"
            "for name in ('sar_layer_norm', 'sar_layer_norm_backward', 'sar_expert_sort', 'sar_expert_dispatch',\n"
            "             'sar_expert_combine', 'sar_expert_combine_backward'):\n"
            "    assert name in dir(sar)\n"
            "    try:\n"
            "        getattr(sar, name)\n"
            "    except ImportError:\n"
            "        continue\n"
            "    raise SystemExit(name)\n"
            "assert not hasattr(sar, 'sar_nothing')\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr + run.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_the_module_is_rebuilt_for_another_torch_or_interpreter(tmp_path):
    """Their files may be older than the module, so times do not tell."""
    out = copy(tmp_path, ())
    build = [sys.executable, str(tmp_path / PACKAGE / "build.py")]
    assert subprocess.run(build, capture_output=True).returncode == 0
    obj, module, key = out / "torch_binding.cpp.obj", out / "_sar_torch.so", out / "torch_binding.key"
    first = [f.stat().st_mtime_ns for f in (obj, module)]
    assert subprocess.run(build, capture_output=True).returncode == 0
    assert [f.stat().st_mtime_ns for f in (obj, module)] == first
    key.write_text(key.read_text().replace("cpython", "another"))
    assert subprocess.run(build, capture_output=True).returncode == 0
    assert all(f.stat().st_mtime_ns > t for f, t in zip((obj, module), first))
