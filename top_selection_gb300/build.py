"""Builds libds_topk.so (the CUDA kernels and the C ABI) in-tree with nvcc for sm_103a, and
_ops.so (the tensor binding over it) with g++ against the installed torch."""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libds_topk.so")
BINDING = os.path.join(HERE, "_ops.so")
BUILT_FOR = os.path.join(HERE, "_ops.built_for")  # the torch and Python that BINDING was built against
BINDING_SOURCE = os.path.join(CSRC, "ds_torch.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("ds_topk.cu", "ds_route.cu", "ds_verify.cu", "ds_cache.cu",
                                           "ds_attend.cu", "ds_experts.cu", "ds_logprobs.cu", "ds_quantise.cu",
                                           "ds_product.cu")]


def deps() -> list:
    """Every file the library is built from: the CUDA sources and headers under csrc/ and
    the public headers (globbed, so a new or edited header always triggers a rebuild)."""
    out = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
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


def _torch_dir():
    """torch's folder, found without importing it; None where torch is not installed (the C ABI
    needs none, and is then all that is built)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_version() -> str:
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"^__version__ *(?::[^=]*)?= *['\"]([^'\"]+)", f.read(), flags=re.M).group(1)


def binding_matches() -> bool:
    """Whether the binding was built against this torch and Python: it uses the C++ interface of one
    torch release, which another need not keep."""
    try:
        with open(BUILT_FOR) as f:
            return f.read() == f"{_torch_version()} {sys.implementation.cache_tag}"
    except OSError:
        return False


def _outputs() -> list:
    return [LIB, BINDING] if _torch_dir() else [LIB]


def up_to_date() -> bool:
    if not all(os.path.exists(o) for o in _outputs()) or (_torch_dir() and not binding_matches()):
        return False
    t = min(os.path.getmtime(o) for o in _outputs())
    return all(os.path.getmtime(d) <= t for d in deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    torch, suffix = _torch_dir(), f".tmp{os.getpid()}"
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="ds_build_") as work:
        # one compiler per source, all at once, then the links
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        cmds = [[_nvcc(), *compile_flags, "-c", "-o", o, s] for s, o in zip(SOURCES, objects)]
        binding = os.path.join(work, "binding.o")
        if torch:
            cuda = os.path.dirname(os.path.dirname(shutil.which(_nvcc()) or "/usr/local/cuda/bin/nvcc"))
            include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                       os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
            cmds.append(["g++", "-O2", "-std=c++17", "-fPIC", *("-I" + d for d in include), "-c", "-o", binding,
                         BINDING_SOURCE])
        if verbose:
            for cmd in cmds:
                print(" ".join(cmd), file=sys.stderr)
        running = [subprocess.Popen(cmd) for cmd in cmds]
        codes = [p.wait() for p in running]
        for cmd, rc in zip(cmds, codes):
            if rc != 0:
                raise subprocess.CalledProcessError(rc, cmd)
        subprocess.run([_nvcc(), *NVCC_FLAGS, "-o", LIB + suffix, *objects], check=True)
        os.replace(LIB + suffix, LIB)
        if torch:  # finds libds_topk.so beside itself
            subprocess.run(["g++", "-shared", "-o", BINDING + suffix, binding, "-L" + os.path.join(torch, "lib"),
                            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + HERE,
                            "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"], check=True)
            if os.path.exists(BUILT_FOR):
                os.remove(BUILT_FOR)
            os.replace(BINDING + suffix, BINDING)
            with open(BUILT_FOR + suffix, "w") as f:
                f.write(f"{_torch_version()} {sys.implementation.cache_tag}")
            os.replace(BUILT_FOR + suffix, BUILT_FOR)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
