"""Build libtg_gemm.so in-tree from csrc/*.cu for sm_100a, and beside it the
Python module _tg_calls from csrc/calls.c, which calls it (where there is a C
compiler and this Python's headers; without it those calls go through ctypes).

    python tiled_dense_gemm_tma_b200/build.py [--force] [--verbose]

Each translation unit is compiled with nvcc (-gencode arch=compute_100a,
code=sm_100a -O3 -lineinfo) into _build/, then linked into a shared library
with the CUDA runtime linked statically.  The driver API entry point used
for tensor-map encoding is looked up at run time, so the library loads on a
machine without a GPU driver (only its compute calls need a device).
"""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libtg_gemm.so")
CALLS = os.path.join(HERE, "_tg_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if not _stale(obj, [src] + _deps()):
        return obj
    cmd = [NVCC] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
    return obj


def _build_calls(force):
    """The module finds the library beside itself, wherever both are moved.  Its
    name carries the interpreter's tag: each Python builds and finds its own."""
    untagged = os.path.join(HERE, "_tg_calls.so")      # what builds before the tag left: any Python finds it
    if os.path.exists(untagged) and untagged != CALLS:
        os.remove(untagged)
    src = os.path.join(CSRC, "calls.c")
    if not force and not _stale(CALLS, [src, os.path.join(INCLUDE, "tg_gemm.h")]):
        return
    tmp = CALLS + f".tmp{os.getpid()}"
    try:
        _compile_calls(src, tmp)
    except (OSError, subprocess.CalledProcessError) as e:
        # no C compiler, or no headers of this Python: the library is all that a call needs
        sys.stderr.write(f"_tg_calls is not built ({e}); its calls go through ctypes, 1.3 us more each\n")
        return
    os.replace(tmp, CALLS)


def _compile_calls(src, out):
    subprocess.run(["gcc", "-O2", "-std=c11", "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-I",
                    sysconfig.get_path("include"), src, "-o", out, "-L", HERE, "-l:libtg_gemm.so",
                    "-Wl,-rpath,$ORIGIN"], check=True)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_library(force, verbose)
    _build_calls(force)
    return OUT


def _build_library(force, verbose):
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if not force and not _stale(OUT, srcs + _deps()):
        return
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
