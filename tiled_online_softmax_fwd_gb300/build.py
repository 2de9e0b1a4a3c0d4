"""Build libfattn.so in-tree (tiled_online_softmax_fwd_gb300/_build/) with nvcc.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into one shared library with the CUDA runtime linked statically and only the
C-ABI symbols exported.  Beside it goes the compiled part of the Python binding
(csrc/binding.cpp), for the interpreter and torch that run the build.

    python -m tiled_online_softmax_fwd_gb300.build [--verbose] [--force]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libfattn.so")
BINDING = os.path.join(BUILD, "fattn_binding.so")

SOURCES = ["fattn_api.cu", "fattn_fwd_sm103.cu", "fattn_bwd_sm103.cu", "fattn_fwd_simt.cu",
           "fattn_rowops.cu", "fattn_rope.cu", "fattn_paged_sm103.cu", "fattn_tree_sm103.cu",
           "fattn_cross_sm103.cu", "fattn_cross_bwd_sm103.cu", "fattn_cross_few.cu",
           "fattn_pages.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
EXPORTS = "{ global: attn_fwd*; attn_bwd*; fattn_*; local: *; };\n"


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found (CUDA 13 toolkit required)")
    return path


def _inputs_newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, "fattn.h")]


def _compile(src: str, verbose: bool, force: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(CSRC, src)] + _headers()
    if not force and not _inputs_newer(obj, deps):
        return obj
    cmd = [nvcc(), *GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj + ".tmp"]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, res.stdout, res.stderr))
    if verbose and (res.stdout or res.stderr):
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(obj + ".tmp", obj)
    return obj


def _run(cmd, what):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, res.stdout, res.stderr))


def _compile_binding(force: bool):
    """binding.cpp for this interpreter and its torch; None if that has no CUDA."""
    import torch
    if torch.version.cuda is None:
        return None
    obj = os.path.join(BUILD, "binding.o")
    src = os.path.join(CSRC, "binding.cpp")
    stamp = obj + ".torch"
    built_for = "%s %s" % (torch.__version__, sys.version)
    if not force and not _inputs_newer(obj, [src, os.path.join(INCLUDE, "fattn.h")]) \
            and os.path.exists(stamp) and open(stamp).read() == built_for:
        return obj
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
          "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
          "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c", src, "-o", obj + ".tmp"],
         "g++ on binding.cpp")
    os.replace(obj + ".tmp", obj)
    with open(stamp, "w") as f:
        f.write(built_for)
    return obj


def _link_binding(obj: str, force: bool):
    import torch
    if not force and not _inputs_newer(BINDING, [obj, LIB]):
        return
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run(["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L", BUILD, "-l:libfattn.so", "-L", lib, "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib],
         "linking the binding")
    os.replace(BINDING + ".tmp", BINDING)


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile and link libfattn.so and the binding; returns the library's path.
    Rebuilds only what changed."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, force)
        objs = list(ex.map(lambda s: _compile(s, verbose, force), SOURCES))
        binding = binding.result()
    if force or _inputs_newer(LIB, objs):
        vmap = os.path.join(BUILD, "exports.map")
        with open(vmap, "w") as f:
            f.write(EXPORTS)
        cmd = [nvcc(), *GENCODE, "-shared", "-cudart", "static", "-o", LIB + ".tmp", *objs,
               "-Xlinker", "--version-script=" + vmap]
        _run(cmd, "link")
        os.replace(LIB + ".tmp", LIB)
    if binding is not None:
        _link_binding(binding, force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(verbose=a.verbose, force=a.force))
