"""Build libexattn.so in-tree with nvcc for sm_103a only.

    python -m exact_attention_67_gb300.build [--force]

Each .cu file is compiled in parallel to an object file, then linked into
exact_attention_67_gb300/_build/libexattn.so; binding.cpp, the Python side of
the paged-cache calls, is compiled by g++ against PyTorch's headers and linked
to it as _build/_exattn_binding.so.  No CMake, one -gencode.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libexattn.so")
BINDING = os.path.join(OUT_DIR, "_exattn_binding.so")
SOURCES = ["api.cu", "fwd.cu", "merge.cu", "bwd.cu", "dq.cu", "decode.cu", "noalloc.cu", "host.cu",
           "paged_api.cu", "rotary.cu", "pages.cu", "paged_decode.cu", "paged_fwd.cu", "paged_merge.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "exattn.h"),
                                                                  os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files if os.path.isfile(f))


def _binding_for() -> str:
    """What the Python module is compiled against; another Python or PyTorch may lay
    its objects out otherwise."""
    import torch
    return f"{sys.implementation.cache_tag} torch {torch.__version__}"


def binding_fits() -> bool:
    """Whether the Python module was built for this Python and PyTorch (its note of
    them lies beside it)."""
    try:
        with open(BINDING + ".for") as f:
            return f.read() == _binding_for()
    except OSError:
        return False


def up_to_date() -> bool:
    return all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime() for f in (LIB, BINDING)) and binding_fits()


def _binding_flags():
    """Compiler and linker flags of binding.cpp: PyTorch's headers and libraries
    (loaded before the module is), Python's headers."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [os.path.join(base, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_flags = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                     "-I", INCLUDE, *[x for i in includes for x in ("-isystem", i)]]
    link_flags = ["-shared", "-L", OUT_DIR, "-lexattn", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(base, "lib"),
                  "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return compile_flags, link_flags


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    cxx = os.environ.get("CXX", "g++")
    binding_obj = os.path.join(OUT_DIR, "binding.o")

    def compile_binding():
        compile_flags, link_flags = _binding_flags()
        cmd = [cxx, *compile_flags, "-c", os.path.join(CSRC, "binding.cpp"), "-o", binding_obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cxx} failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
        return link_flags

    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        bound = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # The library is in place for C callers whatever becomes of the Python side.
    link_flags = bound.result()
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run([cxx, binding_obj, "-o", tmp, *link_flags], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(_binding_for())
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills/shared memory")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra_flags=extra))


if __name__ == "__main__":
    sys.exit(main())
