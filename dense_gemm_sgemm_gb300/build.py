"""Build the CUDA library in-tree: dense_gemm_sgemm_gb300/_build/libgemm_gb300.so.

Every CUDA translation unit under csrc/ is compiled for sm_103a only (tcgen05 and the other
arch-specific features need the `a` target), in parallel, and linked into one shared
library with the static CUDA runtime.  No fast-math: denormals, IEEE division and square
root stay on, which the strict-FP32 path relies on.

With it goes the Python binding of the routed products, _build/_routed.so, compiled against the
installed torch.  The library does not need it: where the binding cannot be built (no torch, a torch
without CUDA, no host C++ compiler) the reason is kept beside it and raised when routed.py is imported.

    python -m dense_gemm_sgemm_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libgemm_gb300.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
BINDING_PATH = os.path.join(OUT_DIR, "_routed.so")
BINDING_SRC = os.path.join(CSRC, "routed_binding.cpp")
BINDING_FOR = os.path.join(OUT_DIR, "_routed.for")      # the torch that the binding was compiled against
BINDING_ERROR = os.path.join(OUT_DIR, "_routed.error")  # why there is none
HEADER = os.path.join(ROOT, "include", "gemm_gb300.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the library needs the CUDA 13 toolkit")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.cuh"))) + [HEADER, os.path.abspath(__file__)]


def _newer(path, deps):
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _read(path):
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _write(path, text):
    tmp = path + f".tmp{os.getpid()}"
    with open(tmp, "w") as f:
        f.write(text)
    os.replace(tmp, path)


def torch_abi() -> str:
    """What a compiled binding depends on: torch's version and C++ ABI, and Python's."""
    try:
        import torch

        return f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, " + str(
            sysconfig.get_config_var("SOABI"))
    except (ImportError, OSError) as e:  # none, or one whose own libraries do not load
        return f"no torch: {e}"


def note_torch() -> None:
    _write(BINDING_FOR, torch_abi())


def built_for() -> str:
    """torch_abi() of the build that made the binding."""
    return _read(BINDING_FOR)


def binding_current() -> bool:
    """Whether the binding on disk is of these sources and of the installed torch."""
    return _newer(BINDING_PATH, [BINDING_SRC, HEADER, os.path.abspath(__file__)]) and built_for() == torch_abi()


def binding_error() -> str:
    """Why the last build made no binding; empty if it did."""
    return _read(BINDING_ERROR).partition("\n")[2]


def _binding_settled() -> bool:
    # a failure is tried again when the sources or torch have changed
    failed = _newer(BINDING_ERROR, [BINDING_SRC, HEADER, os.path.abspath(__file__)])
    return binding_current() or (failed and _read(BINDING_ERROR).startswith(torch_abi() + "\n"))


def up_to_date() -> bool:
    return _newer(LIB_PATH, _deps()) and _binding_settled()


def _compile(nvcc, src, obj, ptxas_verbose):
    cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
           "-c", src, "-o", obj]
    if ptxas_verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, r.returncode, r.stdout + r.stderr


def _compile_binding(nvcc, obj):
    import torch  # an ImportError is kept like a compiler's

    include = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return BINDING_SRC, r.returncode, r.stdout + r.stderr


def _link_binding(obj):
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    # the library by its name, found beside the binding; torch's are loaded by importing torch
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", OUT_DIR, f"-l:{LIB_NAME}",
           "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    note_torch()


def _finish_binding(compiled, obj):
    """Links the binding, or keeps the reason why there is none and leaves no older one behind."""
    try:
        _, rc, log = compiled.result()
        if rc != 0:
            raise RuntimeError(f"compiling the binding failed:\n{log}")
        _link_binding(obj)
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)
        _write(BINDING_ERROR, f"{torch_abi()}\n{e}")
        print(f"the routed products' Python binding was not built: {e}", file=sys.stderr)
    else:
        if os.path.exists(BINDING_ERROR):
            os.remove(BINDING_ERROR)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    anew = force or ptxas_verbose
    if not anew and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding, compiled = os.path.join(OUT_DIR, "routed_binding.o"), None
        if anew or not _binding_settled():
            compiled = ex.submit(_compile_binding, nvcc, binding)
        if anew or not _newer(LIB_PATH, _deps()):
            _build_library(ex, nvcc, ptxas_verbose, quiet)
        if compiled is not None:
            _finish_binding(compiled, binding)
    return LIB_PATH


def _build_library(ex, nvcc, ptxas_verbose, quiet):
    objs, futs = [], []
    for src in _sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        futs.append(ex.submit(_compile, nvcc, src, obj, ptxas_verbose))
    for f in futs:
        src, rc, log = f.result()
        if rc != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{log}")
        if log.strip() and (ptxas_verbose or not quiet):
            print(f"--- {os.path.basename(src)}\n{log}", file=sys.stderr)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    # Static CUDA runtime; driver entry points (tensor-map encoding) are looked up at run
    # time through cudaGetDriverEntryPointByVersion, so the library loads without a driver.
    link = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas, quiet=False))


if __name__ == "__main__":
    main()
