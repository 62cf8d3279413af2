"""Build the CUDA library in-tree: csrc/*.cu -> _build/libw4a16.so (sm_103a).

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library against the shared CUDA runtime (the one PyTorch loads).
``build(checked=True)`` builds the bounds-checked variant instead
(-DW4A16_CHECKED, _build/checked/libw4a16_checked.so): every global access of
its kernels and every place in shared memory that a copy or a product is given
is tested against its buffer first, and one outside sets a bit of the device
error word instead of being used (csrc/common.cuh).
Load it by setting W4A16_LIBRARY to its path before the binding loads the
library. Both also compile csrc/binding.cpp (the Python binding's native part)
with the host compiler against PyTorch's headers. Running ``python -m bit_weight_only_g128_gb300.build [--checked]``
builds by hand.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libw4a16.so")
BUILD_CHECKED = os.path.join(BUILD, "checked")
LIB_CHECKED = os.path.join(BUILD_CHECKED, "libw4a16_checked.so")
BINDING = os.path.join(BUILD, "_binding.so")
BINDING_FOR = BINDING + ".torch"  # the PyTorch version that it was compiled for
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I" + INCLUDE, "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin/ on PATH)")


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(f) for f in files)


def binding_version() -> str:
    """The PyTorch version that _binding.so was compiled for ("" without one)."""
    if not (os.path.exists(BINDING) and os.path.exists(BINDING_FOR)):
        return ""
    with open(BINDING_FOR) as f:
        return f.read()


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp to the CPython module _build/_binding.so
    (against PyTorch's headers, host compiler) if it is not there, older than
    its sources or of another PyTorch; returns its path."""
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if (not force and binding_version() == torch.__version__
            and os.path.getmtime(BINDING) >= max(map(os.path.getmtime, deps))):
        return BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    headers = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    os.makedirs(BUILD, exist_ok=True)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f for h in headers for f in ("-isystem", h)], "-I" + INCLUDE, src, "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for binding.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(torch.__version__)
    return BINDING


def _compile(src: str, obj: str, extra) -> str:
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    return res.stderr


def build(force: bool = False, verbose: bool = False, extra_flags=(), checked: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link libw4a16.so (with
    `checked`, the bounds-checked libw4a16_checked.so); returns its path."""
    out_dir, lib = (BUILD_CHECKED, LIB_CHECKED) if checked else (BUILD, LIB)
    os.makedirs(out_dir, exist_ok=True)
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _deps_mtime():
        build_binding()
        return lib
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(out_dir, os.path.basename(s)[:-3] + ".o") for s in sources]
    extra = list(extra_flags) + (["-DW4A16_CHECKED"] if checked else []) + (["-Xptxas", "-v"] if verbose else [])
    with cf.ThreadPoolExecutor(max_workers=min(os.cpu_count() or 8, len(sources) + 1)) as ex:
        binding = ex.submit(build_binding, force)
        logs = list(ex.map(lambda so: _compile(so[0], so[1], extra), zip(sources, objs)))
        binding.result()
    if verbose:
        for src, log in zip(sources, logs):
            if log.strip():
                print(f"== {os.path.basename(src)}\n{log}", file=sys.stderr)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, checked="--checked" in sys.argv))
