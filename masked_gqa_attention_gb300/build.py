"""Build the CUDA libraries for sm_103a with nvcc, in-tree.

Each translation unit under csrc/ compiles in parallel to an object file;
the objects link into two libraries under masked_gqa_attention_gb300/_lib:
  * libmgqa.so        -- the product library;
  * libmgqa_debug.so  -- the same sources with MGQA_DEBUG: device-side bounds
                         checks, event counters and an injectable pipeline
                         stall (include/masked_gqa_attn_debug.h); test equipment.
csrc/bind.cpp, the Python side of the calls made once per layer and token, goes
into _lib/_mgqa_bind.so beside them (g++ with PyTorch's headers), linked to
libmgqa.so.
The CUDA runtime is linked statically; the driver entry point used for TMA
tensor maps is fetched at run time, so the libraries load on machines
without a GPU.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libmgqa.so")
LIB_DEBUG = os.path.join(OUT_DIR, "libmgqa_debug.so")
BIND = os.path.join(OUT_DIR, "_mgqa_bind.so")
OBJ_DIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]
# variant -> (library, object directory, extra flags)
VARIANTS = {
    "release": (LIB, OBJ_DIR, []),
    "debug": (LIB_DEBUG, os.path.join(OBJ_DIR, "debug"), ["-DMGQA_DEBUG=1"]),
}


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(os.path.dirname(PKG), "include", "*.h"))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _bind_flags():
    """(compile, link) flags of bind.cpp."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tlib = os.path.join(t, "lib")
    return (["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w", *(f"-I{d}" for d in inc)],
            [f"-L{OUT_DIR}", "-l:libmgqa.so", f"-L{tlib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
             "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{tlib}"])


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_bind(obj):
    """bind.cpp to obj; returns the flags of its link."""
    os.makedirs(os.path.dirname(obj), exist_ok=True)
    flags, link = _bind_flags()
    _run(["g++", *flags, "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj], "bind.cpp")
    return link


def build(force: bool = False, verbose: bool = False, extra_flags=(),
          variants=("release", "debug")) -> str:
    """Compile and link the requested variants (both by default), and the Python
    side of the product library with it; returns the product library's path. The
    libraries are in place before a failure of the Python side is raised."""
    todo = [v for v in variants if force or not up_to_date(VARIANTS[v][0])]
    bind = "release" in variants and (force or not up_to_date(BIND))
    if not todo and not bind:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    srcs = _sources()

    def compile_one(job):
        variant, src = job
        _, obj_dir, flags = VARIANTS[variant]
        obj = os.path.join(obj_dir, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *flags, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)} ({variant}):\n"
                               f"{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(f"[{variant}] {os.path.basename(src)}\n{r.stdout}{r.stderr}")
        return obj

    for v in todo:
        os.makedirs(VARIANTS[v][1], exist_ok=True)
    jobs = [(v, src) for v in todo for src in srcs]
    workers = max(1, min(len(jobs) + 1, os.cpu_count() or 8))
    bind_obj = os.path.join(OBJ_DIR, "bind.o")
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        bound = ex.submit(_compile_bind, bind_obj) if bind else None
        objs = list(ex.map(compile_one, jobs))
    for v in todo:
        lib = VARIANTS[v][0]
        vobjs = [o for (vv, _), o in zip(jobs, objs) if vv == v]
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *vobjs, "-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed ({v}):\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if bound:
        link = bound.result()
        tmp = BIND + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, bind_obj, *link], "link of _mgqa_bind.so")
        os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    import sys
    variants = ("release",) if "--release-only" in sys.argv else ("release", "debug")
    print(build(force="--force" in sys.argv, verbose=True, variants=variants,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
