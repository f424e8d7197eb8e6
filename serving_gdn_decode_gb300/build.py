"""Build libgdn_gb300.so (the C-ABI library) in-tree with nvcc for sm_103a,
and the compiled torch binding of the full-attention operators beside it.

Each ``csrc/*.cu`` compiles to an object in parallel, then nvcc links the
shared library next to this file.  ptxas register/spill reports go to
``_build/ptxas.log``.  ``csrc/paged_binding.cpp`` compiles with g++ against the
installed torch's headers; the library itself needs neither, and where torch is
not installed it is all that is built.  Run as
``python -m serving_gdn_decode_gb300.build``.
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
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libgdn_gb300.so")
BINDING = os.path.join(HERE, "_paged_binding.so")
BINDING_SRC = os.path.join(CSRC, "paged_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn_gb300.so")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "gdn.h"),
                                                         os.path.abspath(__file__)]


def _newer(out: str, deps: list[str]) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _binding_up_to_date() -> bool:
    """Whether the binding is there, for this library's header, this Python and this torch."""
    try:
        with open(_stamp_path()) as f:
            stamp = f.read()
    except OSError:
        return False
    return stamp == _binding_stamp() and _newer(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "gdn.h"),
                                                         os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _lib_up_to_date() and (_torch_root() is None or _binding_up_to_date())


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _torch_root() -> str | None:
    import importlib.util
    spec = importlib.util.find_spec("torch")  # its place only: importing it takes seconds
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _stamp_path() -> str:
    return os.path.join(BUILD, "paged_binding.for")


def _binding_stamp() -> str:
    """What a binding is compiled for: one of another Python or torch would not load, or worse, would."""
    import importlib.metadata
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"python {sys.version}\ntorch {version} in {_torch_root()}\n"


def _compile_binding(root: str) -> str:
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "paged_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-I", os.path.join(ROOT, "include"), "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(root: str, obj: str) -> None:
    libs = os.path.join(root, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:" + os.path.basename(LIB), "-L", libs, "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(_stamp_path(), "w") as f:
        f.write(_binding_stamp())


def _build_lib() -> None:
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(16, len(srcs))) as ex:
        results = list(ex.map(_compile, srcs))
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (obj, log), src in zip(results, srcs):
            f.write(f"==== {os.path.basename(src)}\n{log}\n")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart_static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    root = _torch_root()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding, root) if root and (force or not _binding_up_to_date()) else None
        if force or not _lib_up_to_date():
            _build_lib()
    if binding is not None:  # whatever became of it, the library is there
        _link_binding(root, binding.result())
    if verbose:
        print(f"built {LIB}")
        if root is None:
            print("torch is not installed: the full-attention operators are in the library, their torch binding was not built")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
