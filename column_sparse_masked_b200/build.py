"""Builds the CUDA library libflashmask.so in-tree for sm_100a.

Every .cu file under csrc/ is compiled with nvcc
(-gencode arch=compute_100a,code=sm_100a -lineinfo -O3) into an object under
csrc/_build/ and linked into column_sparse_masked_b200/libflashmask.so with
the static CUDA runtime (the library loads on hosts without a GPU driver).

``build(checks=True)`` compiles the same sources with -DFLASHMASK_CHECKS=1
(objects under csrc/_build_checks/) into libflashmask_checks.so: the range
checks of mask values and scheduler indices that report FLASHMASK_ERR_BOUNDS.

``build_binding()`` compiles csrc/binding/paged_binding.cpp (host code, g++,
against torch's and Python's headers) into _paged_binding.so, the marshalling
of the paged-cache calls from Python; ``build()`` brings it up to date as well
where torch is installed.  The C library needs neither (``build_library()``, or
``--library``).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(CSRC, "_build")
LIB = os.path.join(HERE, "libflashmask.so")
BUILD_CHECKS = os.path.join(CSRC, "_build_checks")
LIB_CHECKS = os.path.join(HERE, "libflashmask_checks.so")
BINDING_SRC = os.path.join(CSRC, "binding", "paged_binding.cpp")
BINDING = os.path.join(HERE, "_paged_binding.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps() -> list:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(os.path.dirname(HERE), "include", "flashmask.h")]


def _binding_key() -> str:
    """What the binding is compiled against; it holds this text and refuses to load under another torch."""
    import torch

    return f"paged binding for torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_stale() -> bool:
    """Whether _paged_binding.so is missing, older than its sources or compiled against another torch or Python."""
    header = os.path.join(os.path.dirname(HERE), "include", "flashmask.h")
    newest = max(os.path.getmtime(BINDING_SRC), os.path.getmtime(header))
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < newest:
        return True
    with open(BINDING, "rb") as f:
        return _binding_key().encode() + b"\0" not in f.read()


def build_binding(force: bool = False) -> str:
    """Compiles (if stale) and returns the path of _paged_binding.so."""
    if not force and not binding_stale():
        return BINDING
    import torch

    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DPAGED_BINDING_KEY="{_binding_key()}"', f'-DPAGED_BINDING_TORCH="{torch.__version__}"',
           *(f"-I{d}" for d in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                                os.path.join(cuda, "include"), sysconfig.get_paths()["include"])),
           BINDING_SRC, "-o", tmp, f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"g++ failed: {' '.join(cmd)}")
    os.replace(tmp, BINDING)
    return BINDING


def build_library(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False, checks: bool = False) -> str:
    """Compiles (if stale) and returns the path of libflashmask.so (libflashmask_checks.so with
    checks=True)."""
    build_dir, lib = (BUILD_CHECKS, LIB_CHECKS) if checks else (BUILD, LIB)
    extra = ["-DFLASHMASK_CHECKS=1"] if checks else []
    os.makedirs(build_dir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    dep_mtime = max(os.path.getmtime(d) for d in _deps())
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), dep_mtime):
            cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0 or ptxas_verbose:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if jobs or not os.path.exists(lib):
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, lib)
    return lib


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False, checks: bool = False) -> str:
    """build_library(), and the paged calls' binding where torch is installed."""
    lib = build_library(force, verbose, ptxas_verbose, checks)
    if importlib.util.find_spec("torch") is None:
        sys.stderr.write("torch is not installed: the paged calls' Python binding is not built\n")
    else:
        build_binding(force)
    return lib


if __name__ == "__main__":
    print((build_library if "--library" in sys.argv else build)(
        force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv, checks="--checks" in sys.argv))
