"""Build libsar.so in-tree with nvcc for sm_103a (GB300).

Usage: ``python allreduce_reduction_rank_gb300/build.py [--force] [--verbose-ptxas]``

Each CUDA translation unit is compiled in parallel into an object file under
``_build/`` and the objects are linked into ``_build/libsar.so`` (C ABI,
declared in ``include/sar.h``; the CUDA runtime is linked statically and its
symbols are kept private).  The torch module ``_build/_sar_torch.so``
(``csrc/torch_binding*.cpp``) is compiled at the same time with the host compiler
against the installed torch; the library does not need it, and where torch or
Python's headers are missing it is left out with a note on stderr.  Floating point is compiled without fast-math,
flush-to-zero or contraction so that the binary32 adds are exactly IEEE adds
with gradual underflow.

This file imports nothing from the package, so it runs before the library
exists.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libsar.so")
TORCH_MODULE = os.path.join(OUT, "_sar_torch.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

# Slowest first, so the parallel build finishes sooner.
SOURCES = ["ll_writeback.cu", "ll_fused.cu", "ll_cluster.cu", "ll_cta.cu", "rsag_e4m3b15.cu", "rsag_e4m3b15_acc.cu",
           "ll.cu", "rsag_e4m3fn_acc.cu", "rsag_e4m3fn.cu", "rsag_bf16_acc.cu", "rsag_fp16_acc.cu", "rsag_fp32_acc.cu", "rsag_fp16.cu",
           "rsag_bf16.cu", "rsag_fp32.cu", "layer_norm_bf16.cu", "layer_norm_fp16.cu", "layer_norm_fp32.cu",
           "orthogonalize.cu", "expert_layer.cu", "orthogonalize_small.cu", "layer_norm.cu", "experts.cu", "route.cu", "expert_sort.cu", "convert.cu", "rsag.cu", "sar_api.cu", "operators_api.cu",
           "noalloc.cu"]
# The torch module's; all are compiled again for another interpreter or torch.
BINDING_SOURCES = ["torch_binding.cpp", "torch_binding_block.cpp"]
HEADERS = ["sar_device.cuh", "sar_internal.h", "rsag_kernels.cuh", "ll_coop.cuh", "ll_packets.cuh", "layer_norm.cuh", "layer_norm_ring.cuh", "tensor_core.cuh", "orthogonalize.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-std=c++17", "-lineinfo",
    "-fmad=false", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", INCLUDE,
]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        p = os.path.join(cand, "bin", "nvcc") if cand else ""
        if p and os.path.exists(p):
            return p
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found: libsar needs the CUDA toolkit to build")
    return p


def torch_dir() -> str:
    """The installed torch's directory; empty without one."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else ""


def binding_lacks() -> str:
    """What the torch module needs to be built and is not here; empty where nothing is missing."""
    if not torch_dir():
        return "torch"
    if not os.path.exists(os.path.join(torch_dir(), "include", "c10", "cuda", "CUDAGuard.h")):
        return "torch's CUDA headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return "" if shutil.which("g++") else "g++"


def binding_key() -> str:
    """The interpreter and torch whose headers define what the torch module may assume."""
    with open(os.path.join(torch_dir(), "version.py")) as f:
        return "\n".join([sysconfig.get_config_var("SOABI") or sys.version, torch_dir(), f.read()])


def compile_binding(force: bool) -> list:
    """The torch module's object files; built again for another interpreter or torch."""
    key_path, key = os.path.join(OUT, "torch_binding.key"), binding_key()
    built_for = ""
    if os.path.exists(key_path):
        with open(key_path) as f:
            built_for = f.read()
    headers = [os.path.join(CSRC, "torch_binding.h"), os.path.join(INCLUDE, "sar.h")]

    def compile_one(src: str) -> str:
        path, obj = os.path.join(CSRC, src), os.path.join(OUT, src + ".obj")
        if force or built_for != key or _stale(obj, [path] + headers):
            cuda = os.path.dirname(os.path.dirname(nvcc_path()))
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w", "-I", INCLUDE,
                   "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir(), "include"),
                   "-I", os.path.join(torch_dir(), "include", "torch", "csrc", "api", "include"),
                   "-I", os.path.join(cuda, "include"), "-c", path, "-o", obj + ".tmp"]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"g++ failed on {src}:\n{res.stdout}\n{res.stderr}")
            os.replace(obj + ".tmp", obj)
        return obj

    with ThreadPoolExecutor(len(BINDING_SOURCES)) as ex:
        objs = list(ex.map(compile_one, BINDING_SOURCES))
    with open(key_path, "w") as f:
        f.write(key)
    return objs


def _stale(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    nvcc = nvcc_path()
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "sar.h")]
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src: str) -> str:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OUT, src.replace(".cu", ".o"))
        if force or verbose_ptxas or _stale(obj, [path] + headers):
            cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", path, "-o", obj + ".tmp"]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
            if verbose_ptxas:
                sys.stderr.write(res.stderr)
            os.replace(obj + ".tmp", obj)
        return obj

    with ThreadPoolExecutor(min(len(SOURCES) + 1, (os.cpu_count() or 4) + 1)) as ex:
        lacks = binding_lacks()
        binding = None if lacks else ex.submit(compile_binding, force)
        objs = list(ex.map(compile_one, SOURCES))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + [
            "-Xlinker", "--exclude-libs,ALL", "-Xlinker", "-z,defs", "-Xlinker", "-soname=libsar.so"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    if lacks:
        sys.stderr.write(f"build.py: the torch module is left out: no {lacks}\n")
        return LIB
    binding_objs = binding.result()
    if force or _stale(TORCH_MODULE, binding_objs + [LIB]):
        tmp = TORCH_MODULE + f".tmp{os.getpid()}"
        lib_dir = os.path.join(torch_dir(), "lib")
        cmd = ["g++", "-shared", "-o", tmp] + binding_objs + [LIB, "-L", lib_dir, "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib_dir]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link of the torch module failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, TORCH_MODULE)
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true", help="print registers/spills per kernel")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))


if __name__ == "__main__":
    main()
