"""Compile libq4q.so (the CUDA kernels and the C ABI) for sm_103a, in-tree.

Each .cu file under csrc/ is compiled by nvcc in parallel, then linked into
q4_quantized_matmul_gb300/_build/libq4q.so.  The CUDA runtime is linked
statically so the library only needs the driver at run time.  csrc/q4q_torch.cpp,
the Python side of the MXFP4 calls, becomes _build/_q4q_torch.so beside it where
there is a torch to compile it against; the library itself needs none, at build
time or run time (python q4_quantized_matmul_gb300/build.py).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libq4q.so")
EXT_SRC = os.path.join(CSRC, "q4q_torch.cpp")
EXT = os.path.join(OUT_DIR, "_q4q_torch.so")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "q4q.h")]


def _newer(target: str, sources) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in sources)


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _ext_abi() -> str:
    """What _q4q_torch.so is compiled for: this interpreter and this torch (its version file, read and not imported)."""
    with open(os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "version.py"), encoding="utf-8") as f:
        return "%s\n%s\n%s" % (sys.version, sysconfig.get_config_var("EXT_SUFFIX"), f.read())


def _ext_up_to_date() -> bool:
    """Newer than its sources, and made for the interpreter and torch that are here now: it uses torch's C++ interface,
    which is that of one version."""
    try:
        with open(EXT + ".abi", encoding="utf-8") as f:
            return f.read() == _ext_abi() and _newer(EXT, [EXT_SRC, os.path.join(ROOT, "include", "q4q.h")])
    except OSError:
        return False


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and (not _has_torch() or _ext_up_to_date())


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, r.stdout, r.stderr))


def _compile_ext() -> str:
    """q4q_torch.cpp against this interpreter's torch; the object file."""
    import torch
    from torch.utils import cpp_extension
    includes = cpp_extension.include_paths() + [sysconfig.get_paths()["include"],
                                                os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    obj = os.path.join(OUT_DIR, "q4q_torch.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I" + os.path.join(ROOT, "include"),
          *[a for i in includes for a in ("-isystem", i)], "-c", EXT_SRC, "-o", obj], "g++ for " + EXT_SRC)
    return obj


def _link_ext(obj: str):
    from torch.utils import cpp_extension
    lib = cpp_extension.library_paths()[0]
    tmp = EXT + ".tmp.%d" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + OUT_DIR, "-lq4q", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib,
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"], "link of " + EXT)
    os.replace(tmp, EXT)
    with open(EXT + ".abi", "w", encoding="utf-8") as f:
        f.write(_ext_abi())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        ext = ex.submit(_compile_ext) if _has_torch() else None
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    # the library is there, whatever becomes of the Python side
    if ext is not None:
        _link_ext(ext.result())
    elif verbose:
        print("no torch: %s is not built" % EXT)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
