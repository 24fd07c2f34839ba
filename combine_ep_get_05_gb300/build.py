"""Build libep_gb300.so from csrc/*.cu for sm_103a, in-tree, with plain nvcc.

Each translation unit is compiled in parallel (``nvcc -c``), then the objects
are linked into one shared library with the C ABI of ``include/ep.h``. The
CUDA runtime is linked statically, so the library needs only the driver.

Beside it, csrc/ep_binding.cpp becomes the Python module _ep_binding, compiled
by the host compiler against the installed torch.
"""
from __future__ import annotations

import contextlib
import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libep_gb300.so")
BINDING_SRC = os.path.join(CSRC, "ep_binding.cpp")
BINDING_PATH = os.path.join(BUILD_DIR, "_ep_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    found = shutil.which("nvcc")
    if found:
        return found
    default = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(default):
        return default
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libep_gb300.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(target, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def _library_is_stale() -> bool:
    return _older(LIB_PATH, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "ep.h")])


def _binding_is_stale() -> bool:
    return _older(BINDING_PATH, [BINDING_SRC, os.path.join(INCLUDE, "ep.h")]) or binding_built_for() != _installed()


def _installed() -> str:
    """The interpreter and the torch whose C++ interfaces a binding is compiled against."""
    import torch

    return f"{sysconfig.get_config_var('EXT_SUFFIX')} torch {torch.__version__} {torch.version.git_version}"


def binding_built_for() -> str:
    """What _installed() was when the binding was compiled, "" if that is not known."""
    try:
        with open(BINDING_PATH + ".for") as f:
            return f.read()
    except FileNotFoundError:
        return ""


def check_binding() -> None:
    """Raises unless the binding that is there was built, and for this interpreter and this torch."""
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it first "
                           "(python -m combine_ep_get_05_gb300.build or __graft_entry__.build())")
    if binding_built_for() != _installed():
        raise RuntimeError(f"{BINDING_PATH} was built for [{binding_built_for()}] and this is [{_installed()}]: build it "
                           "again (python -m combine_ep_get_05_gb300.build)")


def is_stale() -> bool:
    return _library_is_stale() or _binding_is_stale()


def host_compiler() -> str:
    found = shutil.which("g++") or shutil.which("c++")
    if not found:
        raise RuntimeError("g++ not found: a host C++ compiler is needed to build _ep_binding.so")
    return found


def _build_binding() -> None:
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    cmd = [host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE,
           "-isystem", inc, "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], BINDING_SRC, "-o", tmp,
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"{host_compiler()} failed on {BINDING_SRC}:\n{proc.stdout}\n{proc.stderr}")
    with contextlib.suppress(FileNotFoundError):
        os.remove(BINDING_PATH + ".for")  # whatever happens next, the old origin does not stay with the new file
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_PATH + ".for", "w") as f:
        f.write(_installed())


def build(force: bool = False, ptxas_info: bool = False, jobs: int | None = None) -> str:
    """Compile and link the library and the binding if any input changed (or force). Returns the library's path."""
    if not (force or ptxas_info or is_stale()):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        proc = subprocess.run([cc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj], capture_output=True, text=True)
        if proc.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{proc.stdout}\n{proc.stderr}")
        return obj, proc.stderr

    with ThreadPoolExecutor(max_workers=jobs or min(8, os.cpu_count() or 1)) as pool:
        binding = pool.submit(_build_binding) if force or _binding_is_stale() else None
        if force or ptxas_info or _library_is_stale():
            results = list(pool.map(compile_one, sources()))
            if ptxas_info:
                with open(os.path.join(BUILD_DIR, "ptxas.txt"), "w") as f:
                    for obj, log in results:
                        f.write(f"== {os.path.basename(obj)}\n{log}\n")
            tmp = LIB_PATH + f".tmp{os.getpid()}"
            proc = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], capture_output=True,
                                  text=True)
            if proc.returncode != 0:
                raise RuntimeError(f"nvcc link failed:\n{proc.stdout}\n{proc.stderr}")
            os.replace(tmp, LIB_PATH)
        if binding is not None:
            binding.result()  # what fails here leaves the library, which does not need it, in place
    return LIB_PATH


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, ptxas_info="--ptxas" in sys.argv))
