"""Build libpagedattn.so (the CUDA library behind include/pa.h) in-tree, and the
binding's C++ calls (``_build/_pa_binding.so``, a CPython extension that reads
torch tensors' fields; g++ and torch's headers).

Each .cu file is compiled for sm_103a by its own nvcc process (in parallel),
then linked into ``paged_kv_decode_cache_gb300/_build/libpagedattn.so``, which
needs neither g++ nor torch (``--library`` builds it alone).
Either part's build is skipped when its file is newer than every source of it
(and, for the binding, was built for this torch and Python).
``-Xptxas -v`` output (registers, spills, shared memory per kernel) is kept
in ``_build/ptxas.log``.
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
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpagedattn.so")
BINDING = os.path.join(BUILD, "_pa_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedattn")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(path: str, deps: list[str]) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + _headers())


def binding_up_to_date() -> bool:
    return _newer(BINDING, glob.glob(os.path.join(CSRC, "*.cpp")) + _headers()) and binding_fits()


def binding_abi() -> str:
    """What the binding is compiled against, besides its sources: this Python and this torch, whose
    headers' inlined functions it holds."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def binding_fits() -> bool:
    """Whether the binding was built for this Python and torch (noted beside it)."""
    try:
        with open(BINDING + ".abi") as f:
            return f.read() == binding_abi()
    except OSError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _extra_flags() -> list[str]:
    """Extra nvcc flags from PA_EXTRA_NVCC_FLAGS (build-time tuning, e.g. -DPA_TC_NK=2)."""
    return os.environ.get("PA_EXTRA_NVCC_FLAGS", "").split()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xptxas", "-v", "--expt-relaxed-constexpr", *_extra_flags(), "-I", INCLUDE, "-c", src,
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    return obj, r.stderr


def _compile_binding() -> None:
    """The binding's C++ calls (csrc/pa_binding.cpp) against this machine's torch."""
    import torch
    import torch.utils.cpp_extension as ext
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           os.path.join(CSRC, "pa_binding.cpp"), "-o", tmp,
           *[f"-I{d}" for d in ext.include_paths() + [sysconfig.get_paths()["include"]]],
           *[f"-L{d}" for d in ext.library_paths()], "-ltorch_python", "-ltorch_cpu", "-lc10", "-ldl",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and the binding, at the same time; a binding that does not compile raises after the
    library has been built."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_binding, force)
        build_library(force, verbose)
        binding.result()
    return LIB


def build_binding(force: bool = False) -> str:
    if force or not binding_up_to_date():
        os.makedirs(BUILD, exist_ok=True)
        _compile_binding()
        with open(BINDING + ".abi", "w") as f:
            f.write(binding_abi())
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and library_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        results = list(ex.map(_compile, srcs))
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for _, log in results:
            f.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-Xlinker", f"-rpath,{cuda_lib}",
           "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    (build_library if "--library" in sys.argv else build)(force="--force" in sys.argv, verbose=True)
