"""Build in-tree: csrc/*.cu -> libvit_block.so (sm_103a only), the CUDA library, and
csrc/binding.cpp -> _serving.<torch>.<python>.so, the Python marshalling of its serving stages.

Each translation unit is compiled in parallel, with nvcc or g++, then linked next to this
file. A rebuild happens only when a source or header is newer than what is built. The binding
has torch's and Python's object layouts compiled in, so its name holds the build of torch and the
interpreter's tag, and no other is loaded. The library needs nvcc alone; the binding needs torch with its CUDA headers and a C++ compiler, and where they
are missing it is left out with a notice. Usage:
``python -m vision_transformer_encoder_gb300.build``.
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

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libvit_block.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

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
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + _binding_deps()[1:]


def _binding_deps():
    return [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _torch_dir():
    # torch is only located, not imported
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def binding_path():
    """Where the binding for this torch and this interpreter is, or is to be, built; None without torch."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            text = f.read()
    except OSError:
        text = ""
    found = [re.search(r"^%s\b.*?=\s*['\"]([^'\"]+)" % name, text, re.M) for name in ("__version__", "git_version")]
    torch_build = "-".join(re.sub(r"[^\w.+]", "_", m.group(1))[:24] for m in found if m) or "unknown"
    return os.path.join(HERE, "_serving.torch-%s%s" % (torch_build, sysconfig.get_config_var("EXT_SUFFIX")))


def binding_toolchain():
    """(directory of torch, C++ compiler) that the binding is built with, or what is missing, as text."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return "torch is not installed"
    for part in ("include/torch/csrc/Dtype.h", "include/c10/cuda/CUDAGuard.h", "lib/libtorch_cuda.so"):
        if not os.path.exists(os.path.join(torch_dir, part)):
            return "torch has no %s" % part
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h is missing"
    cxx = os.environ.get("CXX") or "g++"
    if shutil.which(cxx) is None:
        return "%s is not found" % cxx
    return torch_dir, cxx


def _library_up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def _binding_up_to_date() -> bool:
    return isinstance(binding_toolchain(), str) or _newer(binding_path(), _binding_deps())


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


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
        path = binding_path()
        tmp = path + ".%d.tmp" % os.getpid()
        run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", include,
             "-I", os.path.join(include, "torch", "csrc", "api", "include"),
             "-I", os.path.join(os.path.dirname(os.path.dirname(cc)), "include"),
             "-I", sysconfig.get_paths()["include"], BINDING_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"),
             "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "%s failed on %s" % (cxx, BINDING_SRC))
        os.replace(tmp, path)

    tools = binding_toolchain()
    with cf.ThreadPoolExecutor(max_workers=min(len(_sources()) + 1, os.cpu_count() or 4)) as ex:
        binding = None
        if isinstance(tools, str):
            print("the Python binding of the serving stages is left out: %s" % tools, file=sys.stderr)
        elif force or not _binding_up_to_date():
            binding = ex.submit(build_binding, *tools)
        if force or not _library_up_to_date():
            # the library stands whatever becomes of the binding
            objs = list(ex.map(compile_one, _sources()))
            tmp = LIB_PATH + ".%d.tmp" % os.getpid()
            run([cc] + ARCH + ["-shared", "-o", tmp] + objs, "link failed")
            os.replace(tmp, LIB_PATH)
        if binding is not None:
            binding.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
