"""Build the gfx950 shared library in-tree with hipcc (no torch involved).

    python block_scaled_fp4_group_amd/build.py

(run as a script: importing the package itself needs the built library)

Each HIP source compiles to its own object in parallel (the GEMM files hold
many kernel instantiations), then one link step writes libmoefp4.so.  The
Python side of the attention calls (csrc/calls.cpp, plain CPython) becomes
_calls.<this Python's tag>.so, linked to it.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmoefp4.so")
CALLS = os.path.join(PKG, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))   # this Python's own
OBJ_DIR = os.path.join(PKG, "_build")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "hipcc"


def sources() -> list:
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.hip")))


def compile_command(src: str, obj: str) -> list:
    return [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wno-unused-command-line-argument",
            "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"), src, "-o", obj]


def link_command(objs: list, out: str) -> list:
    return [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", *objs, "-o", out]


def calls_command(out: str) -> list:
    """Host code only, by the compiler that builds the rest (the HIP header gives the stream's type)."""
    python = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")):
        raise RuntimeError(f"calls.cpp needs Python's headers, and {python}/Python.h is not there")
    rocm = os.path.dirname(os.path.dirname(hipcc())) if os.path.sep in hipcc() else "/opt/rocm"
    return [hipcc(), "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
            "-I", python, "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"),
            os.path.join(PKG, "csrc", "calls.cpp"), "-o", out, "-L", PKG, "-lmoefp4", "-Wl,-rpath,$ORIGIN"]


def _run(cmd: list) -> tuple:
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l and l.strip()]
    return r.returncode, msgs


def build(verbose: bool = True, jobs: int = 0) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sources()
    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-4] + ".o") for s in srcs]
    jobs = jobs or max(1, min(len(srcs), os.cpu_count() or 4, 16))
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        results = list(ex.map(_run, [compile_command(s, o) for s, o in zip(srcs, objs)]))
    failed = False
    for src, (rc, msgs) in zip(srcs, results):
        if rc != 0:
            failed = True
            sys.stderr.write(f"hipcc failed on {os.path.basename(src)}:\n" + "\n".join(msgs) + "\n")
        elif msgs and verbose:
            print("\n".join(msgs))
    if failed:
        raise RuntimeError("hipcc failed")
    tmp = LIB + ".tmp"
    rc, msgs = _run(link_command(objs, tmp))
    if rc != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"link failed with exit code {rc}")
    # a kernel template whose host-side instantiation clang silently drops
    # leaves its launch stub undefined: the link succeeds and loading fails
    undef = subprocess.run(["nm", "-u", tmp], capture_output=True, text=True).stdout
    stubs = [l.split()[-1] for l in undef.splitlines() if "__device_stub__" in l]
    if stubs:
        raise RuntimeError("kernel launch stubs left undefined (host-side instantiation failed): " + ", ".join(stubs[:4]))
    os.replace(tmp, LIB)
    tmp = CALLS + ".tmp"
    rc, msgs = _run(calls_command(tmp))
    if rc != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"the compiler failed on calls.cpp with exit code {rc}")
    os.replace(tmp, CALLS)
    untagged = os.path.join(PKG, "_calls.so")
    if CALLS != untagged and os.path.exists(untagged):                # of before the tag: any Python would load it
        os.remove(untagged)
    if verbose:
        print(f"built {LIB} from {len(srcs)} sources, {CALLS}", flush=True)
    return LIB


if __name__ == "__main__":
    build()
