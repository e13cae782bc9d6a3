"""Builds the CUDA library libmoe_b200.so in-tree for sm_100a, and the Python
binding of its attention operators (_attn_binding, against the installed torch).

    python bit_dequant_expert_b200/build.py [--force] [--jobs N] [--ptxas-verbose]

Each .cu under csrc/ is compiled separately (in parallel) and linked into one
shared library with the CUDA runtime linked statically, so the library only
needs the NVIDIA driver at run time.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
OUT = os.path.join(HERE, "libmoe_b200.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_attn_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_FOR = os.path.join(BUILD, "attn_binding.built_for")   # what the module beside it was built for

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
    "-I", INCLUDE,
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def stale() -> bool:
    if not os.path.exists(OUT):
        return True
    t = os.path.getmtime(OUT)
    return any(os.path.getmtime(p) > t for p in sources() + _deps())


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def binding_for() -> str:
    """What the extension module's binary interface hangs on besides its sources: Python, torch (which one and where) and
    the compiler."""
    cxx = subprocess.check_output([_cxx(), "--version"], text=True).splitlines()[0]
    return "\n".join((sys.version, importlib.metadata.version("torch"), _torch_dir(), cxx)) + "\n"


def binding_stale() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_FOR):
        return True
    with open(BINDING_FOR) as f:
        if f.read() != binding_for():
            return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(p) > t for p in (BINDING_SRC, os.path.join(INCLUDE, "attn_b200.h")))


def build_binding() -> None:
    """The extension module: host code only, linked to the library beside it and to torch's own libraries."""
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    libs = os.path.join(torch_dir, "lib")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    subprocess.check_call(
        [_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", BINDING_SRC, "-o", tmp, "-I", INCLUDE,
         "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
         "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
         "-L", HERE, "-l:libmoe_b200.so", "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
         "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs], env=_env())
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(binding_for())


def _env() -> dict:
    """nvcc's temporary files go to a folder inside the repository."""
    tmpdir = os.path.join(BUILD, "tmp")
    os.makedirs(tmpdir, exist_ok=True)
    return dict(os.environ, TMPDIR=tmpdir)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
    subprocess.check_call(cmd, env=_env())
    return obj


def build(force: bool = False, jobs: int | None = None, extra: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force or stale():
        _build_library(jobs, extra)
    if force or binding_stale():
        build_binding()
    return OUT


def _build_library(jobs: int | None, extra: list[str] | None) -> None:
    extra = extra or []
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = OUT + ".tmp.%d" % os.getpid()
    subprocess.check_call([nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp] + objs,
                          env=_env())
    os.replace(tmp, OUT)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--jobs", type=int, default=None)
    ap.add_argument("--ptxas-verbose", action="store_true")
    args = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if args.ptxas_verbose else []
    print(build(force=args.force or args.ptxas_verbose, jobs=args.jobs, extra=extra))


if __name__ == "__main__":
    main(sys.argv[1:])
