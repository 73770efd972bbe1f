"""Builds libcr.so, the CUDA library of this package, for sm_103a (GB300).

Each translation unit is compiled in parallel with nvcc, then linked into a
shared library next to this file (``_build/libcr.so``). Beside it goes
``_build/cr_model_binding.so``, the Python side of the model operators, which
is host code against PyTorch's headers. The flags keep every
floating-point operation what the source says: no FMA contraction, no
flush-to-zero, IEEE division and square root, never --use_fast_math. (The
convolution and the scan ask for fused multiply-adds and for the approximate
exponential and reciprocal by name.)
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libcr.so")
BINDING_SRC = os.path.join(CSRC, "model_binding.cpp")
BINDING = os.path.join(OUT_DIR, "cr_model_binding.so")
BINDING_STAMP = BINDING + ".stamp"  # what it was built against
SOURCES = ["cr_api.cu", "cr_calibrate.cu", "cr_chain.cu", "cr_conv.cu", "cr_embedding.cu",
           "cr_host_batched.cu", "cr_launch.cu", "cr_noalloc.cu", "cr_reduce.cu",
           "cr_reduce_policy.cu", "cr_scan.cu", "cr_selective_scan.cu",
           "cr_selective_scan_backward.cu"]
HEADERS = ["cr_chain.h", "cr_chain_map.h", "cr_device.cuh", "cr_launch.h", "cr_model.cuh",
           "cr_plan.h", "cr_scan.h", "cr_selective_scan.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--fmad=false", "-ftz=false", "-prec-div=true",
    "-prec-sqrt=true", "-Xcompiler", "-fPIC", "-Xcompiler", "-fno-fast-math",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcr")
    return cand


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src] + [os.path.join(CSRC, h) for h in HEADERS] + [
        os.path.join(ROOT, "include", "cr.h"), __file__]
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_command(nvcc: str, out: str) -> list:
    """g++ on the binding, with PyTorch's headers and libraries found without
    importing it."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [os.path.join(ROOT, "include"), os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            *("-I" + d for d in include), BINDING_SRC, "-o", out,
            "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def _binding_stamp(command: list) -> str:
    """The versions whose ABI the binding has, and how it was compiled."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "\n".join([sys.version, f.read(), *command])


def _binding_stale(stamp: str) -> bool:
    if _stale(BINDING, BINDING_SRC) or not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != stamp


def build(force: bool = False, verbose: bool = False, defines=(), out_dir: str | None = None) -> str:
    """Compiles the sources (those changed since their object, or all with
    force) and links the library; returns its path. `defines` ("NAME=value"
    strings) override the decomposition knobs of the sources (run lengths,
    tiles a block, fill blocks), which change no result; a build with
    defines goes to its own out_dir and is always complete."""
    out = OUT_DIR if out_dir is None else out_dir
    if defines and out_dir is None:
        raise ValueError("a build with overridden knobs needs its own out_dir")
    lib = os.path.join(out, "libcr.so")
    os.makedirs(out, exist_ok=True)
    nvcc = _nvcc()
    flags = NVFLAGS + ["-D" + d for d in defines]
    force = force or bool(defines)
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(out, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, s):
            jobs.append([nvcc, *flags, "-c", s, "-o", o])
    link = bool(jobs)
    new_binding = None
    stamp = _binding_stamp(_binding_command(nvcc, BINDING))
    if out_dir is None and (force or _binding_stale(stamp)):
        new_binding = BINDING + ".tmp.%d" % os.getpid()
        jobs.append(_binding_command(nvcc, new_binding))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for r in ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs):
                if verbose or r.returncode:
                    print(r.stdout + r.stderr)
                if r.returncode:
                    raise RuntimeError("compilation failed: " + " ".join(r.args))
    if new_binding is not None:
        os.replace(new_binding, BINDING)
        with open(BINDING_STAMP, "w") as f:
            f.write(stamp)
    if force or link or not os.path.exists(lib):
        tmp = lib + ".tmp.%d" % os.getpid()
        subprocess.run([nvcc, *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs], check=True)
        os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
