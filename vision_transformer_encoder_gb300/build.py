"""Build in-tree: csrc/*.cu -> libvit_block.so (sm_103a only), the CUDA library, and
csrc/binding.cpp -> _serving.so, the Python marshalling of its serving stages.

Each translation unit is compiled in parallel, with nvcc or g++, then linked next to this
file. A rebuild happens only when a source or header is newer than what is built. The library
needs nvcc alone; the binding needs torch with its CUDA headers and a C++ compiler, and where they
are missing it is left out with a notice. Usage:
``python -m vision_transformer_encoder_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libvit_block.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(HERE, "_serving.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _newer_than_deps(path) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in _deps())


def binding_toolchain():
    """(directory of torch, C++ compiler) that the binding is built with, or what is missing, as text. torch is
    only located, not imported."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return "torch is not installed"
    torch_dir = list(spec.submodule_search_locations)[0]
    for part in ("include/torch/csrc/Dtype.h", "include/c10/cuda/CUDAGuard.h", "lib/libtorch_cuda.so"):
        if not os.path.exists(os.path.join(torch_dir, part)):
            return "torch has no %s" % part
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h is missing"
    cxx = os.environ.get("CXX") or "g++"
    if shutil.which(cxx) is None:
        return "%s is not found" % cxx
    return torch_dir, cxx


def up_to_date() -> bool:
    return _newer_than_deps(LIB_PATH) and (isinstance(binding_toolchain(), str) or _newer_than_deps(BINDING_PATH))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("%s:\n%s%s" % (what, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        run([cc] + NVCC_FLAGS + ["-c", src, "-o", obj], "nvcc failed on %s" % src)
        return obj

    def build_binding(torch_dir, cxx):
        # torch's libraries are in the process before the module is loaded
        include = os.path.join(torch_dir, "include")
        tmp = BINDING_PATH + ".%d.tmp" % os.getpid()
        run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", include,
             "-I", os.path.join(include, "torch", "csrc", "api", "include"),
             "-I", os.path.join(os.path.dirname(os.path.dirname(cc)), "include"),
             "-I", sysconfig.get_paths()["include"], BINDING_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"),
             "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "%s failed on %s" % (cxx, BINDING_SRC))
        os.replace(tmp, BINDING_PATH)

    srcs = _sources()
    tools = binding_toolchain()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = None if isinstance(tools, str) else ex.submit(build_binding, *tools)
        objs = list(ex.map(compile_one, srcs))
        # the library stands whatever becomes of the binding
        tmp = LIB_PATH + ".%d.tmp" % os.getpid()
        run([cc] + ARCH + ["-shared", "-o", tmp] + objs, "link failed")
        os.replace(tmp, LIB_PATH)
        if binding is None:
            print("the Python binding of the serving stages is left out: %s" % tools, file=sys.stderr)
        else:
            binding.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
