"""Builds libh3blk.so (all CUDA sources under csrc/) in-tree for sm_100a, and
_fp4_torch.so (csrc/fp4_torch.cpp, a Python module over it for torch tensors).

    python joint_video_audio_b200/build.py [--force] [--verbose]

Objects go to _build/ at the repository root; the shared library is written
next to this file. nvcc cross-compiles, so no GPU is needed to build.
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
from importlib.util import find_spec

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libh3blk.so")
MODULE = os.path.join(PKG, "_fp4_torch.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                 "-I", INCLUDE, "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libh3blk")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(f for d, ext in ((CSRC, "*.cuh"), (CSRC, "*.h"), (INCLUDE, "*.h")) for f in glob.glob(os.path.join(d, ext)))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose):
    obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [nvcc()] + CFLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
    return obj


def _module_stamp(torch):
    """What the module is built with: which Python, which torch and where."""
    with open(os.path.join(torch, "version.py")) as f:
        return "\n".join([str(sysconfig.get_config_var("SOABI")), sys.version, torch, f.read()])


def _build_module(force):
    src = os.path.join(CSRC, "fp4_torch.cpp")
    torch = os.path.dirname(find_spec("torch").origin)
    # dates do not tell one environment from another: what was built with is kept
    # beside the objects and compared
    stamp, stamp_file = _module_stamp(torch), os.path.join(OBJDIR, "_fp4_torch.stamp")
    if not force and os.path.exists(stamp_file) and not _stale(MODULE, [src] + _headers()):
        with open(stamp_file) as f:
            if f.read() == stamp:
                return
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = MODULE + ".tmp"
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", src, "-o", tmp]
    cmd += [f for d in inc for f in ("-I", d)]
    cmd += ["-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10",
            "-L", PKG, "-l:libh3blk.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(stamp_file):  # (a stamp never stands beside another module than its own)
        os.remove(stamp_file)
    os.replace(tmp, MODULE)
    with open(stamp_file, "w") as f:
        f.write(stamp)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles every csrc/*.cu, links libh3blk.so and the module over it; returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(OBJDIR, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_module(force)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
