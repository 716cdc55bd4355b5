"""Builds libds_topk.so (the CUDA kernels and the C ABI) in-tree with nvcc for sm_103a."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libds_topk.so")
SOURCES = [os.path.join(CSRC, f) for f in ("ds_topk.cu", "ds_route.cu", "ds_verify.cu", "ds_cache.cu",
                                           "ds_attend.cu")]


def deps() -> list:
    """Every file the library is built from: the CUDA sources and headers under csrc/ and
    the public headers (globbed, so a new or edited header always triggers a rebuild)."""
    out = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh", ".h"))]
    out += [os.path.join(INCLUDE, f) for f in sorted(os.listdir(INCLUDE)) if f.endswith(".h")]
    out.append(os.path.abspath(__file__))
    return out

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "-Xcompiler", "-fPIC", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    # one nvcc per source, all at once, then a link
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="ds_build_") as work:
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        cmds = [[_nvcc(), *compile_flags, "-c", "-o", o, s] for s, o in zip(SOURCES, objects)]
        if verbose:
            for cmd in cmds:
                print(" ".join(cmd), file=sys.stderr)
        running = [subprocess.Popen(cmd) for cmd in cmds]
        codes = [p.wait() for p in running]
        for cmd, rc in zip(cmds, codes):
            if rc != 0:
                raise subprocess.CalledProcessError(rc, cmd)
        subprocess.run([_nvcc(), *NVCC_FLAGS, "-o", tmp, *objects], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
