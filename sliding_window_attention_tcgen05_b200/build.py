"""Builds libvx.so in-tree with nvcc for sm_100a.

    python sliding_window_attention_tcgen05_b200/build.py          # incremental
    python sliding_window_attention_tcgen05_b200/build.py --force

(Run it as a script: importing the package itself needs the built library.)

Each csrc/*.cu is compiled to _build/<name>.o (rebuilt when it or any header
is newer than its object) and the objects are linked into
sliding_window_attention_tcgen05_b200/libvx.so with a static CUDA runtime.
csrc/bind.cpp (the paged-cache wrappers' marshalling, against PyTorch's C++
headers) becomes sliding_window_attention_tcgen05_b200/_bind.so, which calls
into libvx.so; it is rebuilt for another torch or Python too.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libvx.so")
BIND = os.path.join(PKG, "_bind.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                     "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(src: str, obj: str, hdr_mtime: float) -> bool:
    if not os.path.exists(obj):
        return True
    om = os.path.getmtime(obj)
    return os.path.getmtime(src) > om or hdr_mtime > om


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_mtime = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    cc = nvcc()
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        if force or ptxas_info or _stale(s, o, hdr_mtime):
            cmd = [cc] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", s, "-o", o]
            jobs.append((s, cmd))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def run(job):
        src, cmd = job
        if verbose:
            print(" ".join(cmd), flush=True)
        p = subprocess.run(cmd, capture_output=True, text=True)
        return src, p

    failed = []
    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for src, p in ex.map(run, jobs):
            out = (p.stdout or "") + (p.stderr or "")
            if out.strip() and (verbose or ptxas_info or p.returncode != 0):
                print(f"--- {os.path.basename(src)}\n{out}", flush=True)
            if p.returncode != 0:
                failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(f) for f in failed))
    lib_stale = force or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs)
    if lib_stale:
        cmd = [cc] + ARCH + ["-shared", "-o", LIB] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError("link failed:\n" + p.stdout + p.stderr)
    build_bind(force=force, verbose=verbose)
    return LIB


def _bind_abi() -> str:
    """What _bind.so is tied to beside its sources."""
    return f"torch {importlib.metadata.version('torch')}, {sysconfig.get_config_var('EXT_SUFFIX')}\n"


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """_bind.so; needs libvx.so."""
    src = os.path.join(CSRC, "bind.cpp")
    hdr = os.path.getmtime(os.path.join(ROOT, "include", "vx.h"))
    stamp, abi = os.path.join(BUILD, "_bind.abi"), _bind_abi()
    built_for = open(stamp).read() if os.path.exists(stamp) else None
    if not force and built_for == abi and not _stale(src, BIND, hdr):
        return BIND

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_bind",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, src, "-o", BIND, "-L", lib, "-L", PKG,
           "-l:libvx.so", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("bind.cpp failed:\n" + p.stdout + p.stderr)
    with open(stamp, "w") as f:
        f.write(abi)
    return BIND


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / smem per kernel")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    sys.exit(main())
