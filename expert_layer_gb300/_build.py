"""Builds libmoe_gb300.so in-tree with nvcc for sm_103a, and the Python binding
of the attention functions (_attn_binding.so) with the host compiler.  The
library needs nvcc alone: where the binding cannot be built (no g++, or no
headers of PyTorch or Python), the build warns and those functions raise.

Each .cu file under csrc/ compiles to its own object (in parallel); the
objects link into expert_layer_gb300/libmoe_gb300.so.  A file is recompiled
when it or any header is newer than its object.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(PKG, "_attn_binding.so")
CXX = "g++"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_gb300.so")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "moe.h"))
    return hs


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def build_binding(verbose: bool = False) -> str:
    """Compile the extension module of the attention functions (host C++ against
    this PyTorch's headers); returns its path.  Rebuilt when its source, the
    C header, PyTorch or Python changed; put in place whole, so that a process
    that has the old one mapped keeps it."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "attn_binding.cpp")
    out, part = BINDING, f"{BINDING}.{os.getpid()}.so"
    made_for = os.path.join(BUILD, "attn_binding.for")
    this = f"{torch.__version__} {torch.__file__} {sysconfig.get_config_var('EXT_SUFFIX')}"
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(ROOT, "include", "moe.h")))
    if os.path.exists(out) and os.path.getmtime(out) >= newest and os.path.exists(made_for):
        with open(made_for) as f:
            if f.read() == this:
                return out
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(at, "include"),
           "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), src, "-o", part,
           "-L", os.path.join(at, "lib"), "-lc10", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{CXX} failed for {src}:\n{r.stdout}\n{r.stderr}")
        os.replace(part, out)
    except (RuntimeError, OSError):
        for f in (part, out):             # one for other sources or another PyTorch is not left behind
            if os.path.exists(f):
                os.remove(f)
        raise
    with open(made_for, "w") as f:
        f.write(this)
    return out


def build(verbose: bool = False, extra_flags: list[str] | None = None, build_dir: str | None = None,
          lib_path: str | None = None) -> str:
    """Compile and link the library; returns its path.  ``extra_flags`` go to
    every nvcc compile (e.g. ["-DMOE_DEBUG_BOUNDS"] for the index-checking
    build, which then needs its own ``build_dir`` and ``lib_path``)."""
    nvcc = _nvcc()
    BUILD = build_dir or globals()["BUILD"]
    LIB = lib_path or globals()["LIB"]
    os.makedirs(BUILD, exist_ok=True)
    newest_hdr = max(os.path.getmtime(h) for h in _headers())
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), newest_hdr):
            return obj
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = None if lib_path else ex.submit(build_binding, verbose)
        objs = list(ex.map(compile_one, sources()))
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if binding is not None:
        try:
            binding.result()
        except (RuntimeError, OSError, ImportError) as e:
            warnings.warn(f"the attention functions are not available, their binding was not built: {e}", stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
