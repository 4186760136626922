"""Build libhata.so in-tree with nvcc for sm_100a.

    python hash_aware_top_b200/build.py [--force] [--verbose] [--ptxas-v]

(run as a script: importing the package itself loads the built library)

Compiles every hash_aware_top_b200/csrc/*.cu to an object under _build/ and
links them into hash_aware_top_b200/libhata.so (CUDA runtime linked
statically), then the benchmark's loop (libhata_e2e.so) and the native half of
the binding (_serving.<ABI>.so, g++ against the headers of the installed torch).
Rebuilds only when a source or header is newer than the library; the native
half also when torch, the interpreter or the compiler is another.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import json
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "libhata")
LIB = os.path.join(PKG, "libhata.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    srcs = _sources()
    hdrs = _headers()
    if not force and not _stale(LIB, srcs + hdrs) and not _stale(E2E_LIB, [E2E_SRC, LIB]):
        build_binding(False, verbose)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        if force or _stale(obj, [src] + hdrs):
            cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_e2e(cc, flags, verbose)
    build_binding(force, verbose)
    return LIB


E2E_SRC = os.path.join(PKG, "e2e", "hata_e2e.cu")
E2E_LIB = os.path.join(PKG, "libhata_e2e.so")


def build_e2e(cc, flags, verbose=False):
    """The benchmark's end-to-end loop (native, calling libhata.so's C ABI)."""
    obj = os.path.join(BUILD, "hata_e2e.o")
    cmds = [[cc, *ARCH, *flags, "-c", E2E_SRC, "-o", obj],
            [cc, *ARCH, "-shared", "-o", E2E_LIB + ".tmp", obj, "-L" + PKG, "-lhata", "-Xlinker", "-rpath=$ORIGIN"]]
    for cmd in cmds:
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"e2e driver build failed:\n{r.stdout}\n{r.stderr}")
    os.replace(E2E_LIB + ".tmp", E2E_LIB)


BINDING_SRC = os.path.join(PKG, "binding", "serving.cpp")
BINDING_LIB = os.path.join(PKG, "_serving" + sysconfig.get_config_var("EXT_SUFFIX"))  # an interpreter finds its own alone
BINDING_STAMP = os.path.join(PKG, "_serving.json")  # what it was built for


def binding_built_for() -> str:
    """What the native half of the binding is tied to; it is compiled in and compared when the package is imported."""
    import torch

    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def build_binding(force=False, verbose=False):
    """The native half of the Python binding.  It calls the C ABI and torch's, so it is rebuilt when a header changes, and for
    another torch, interpreter or compiler than the stamp beside it names."""
    import torch  # its headers, its ABI

    base = os.path.dirname(torch.__file__)
    key = [binding_built_for(), base, sysconfig.get_paths()["include"], os.environ.get("CXX", "g++")]
    try:
        with open(BINDING_STAMP) as f:
            same = json.load(f) == key
    except (OSError, ValueError):
        same = False
    if not force and same and not _stale(BINDING_LIB, [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return
    tmp = BINDING_LIB + ".tmp"
    cmd = [key[-1], "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DHATA_BUILT_FOR="{key[0]}"', "-I", INCLUDE,
           "-I", os.path.join(base, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
           BINDING_SRC, "-o", tmp, "-L" + PKG, "-lhata", "-L" + os.path.join(base, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding build failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_LIB)
    with open(BINDING_STAMP, "w") as f:
        json.dump(key, f)
    untagged = os.path.join(PKG, "_serving.so")  # as builds made it before, for any interpreter to find
    if os.path.exists(untagged):
        os.remove(untagged)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/shared-memory usage")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_v else None
    print(build(force=a.force or a.ptxas_v, verbose=a.verbose or a.ptxas_v, extra_flags=extra))


if __name__ == "__main__":
    sys.exit(main())
