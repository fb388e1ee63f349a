"""Builds libdsa_gb300.so in-tree with nvcc for sm_103a (one translation unit
per .cu file, compiled in parallel, then linked; no cmake, no torch), and the
module that marshals the serving calls' tensors (_binding.so, g++ against
PyTorch's and Python's headers; without those the Python code does its work)."""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdsa_gb300.so")
BINDING, BINDING_SRC = os.path.join(PKG, "_binding.so"), os.path.join(CSRC, "binding.cpp")
SOURCES = ["api.cu", "topk.cu", "simt.cu", "indexer_tc.cu", "attn_fwd_tc.cu", "static_ws.cu",
           "bwd_tc.cu", "kl_tc.cu", "indexer_fp8.cu", "cache.cu", "tree_attn.cu", "tree_attn_tc.cu",
           "beam.cu", "rope.cu", "sample.cu", "accept.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsa_gb300.so")


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src, os.path.join(CSRC, "dsa_common.cuh"), os.path.join(CSRC, "tree_attn.cuh"), os.path.join(CSRC, "bound.h"),
            os.path.join(ROOT, "include", "dsa.h"), __file__]
    return any(os.path.getmtime(d) > os.path.getmtime(obj) for d in deps)


def binding_stamp(torch_version: str) -> str:
    """What _binding.so is made of: the package loads only one that carries the present stamp."""
    h = hashlib.sha256(f"{torch_version} {sys.version}".encode())
    for path in (BINDING_SRC, os.path.join(ROOT, "include", "dsa.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def _drop_binding() -> None:
    """An old module must not outlive the sources it was made of."""
    for path in (BINDING, BINDING + ".tmp"):
        if os.path.exists(path):
            os.remove(path)


def _binding_job(nvcc: str, force: bool):
    """The command that builds _binding.so, or None: up to date, or it cannot be built (then there is none)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        _drop_binding()
        return None
    torch, python = os.path.dirname(spec.origin), sysconfig.get_paths()["include"]
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"), python,
           cuda, os.path.join(ROOT, "include")]
    deps = [BINDING_SRC, os.path.join(ROOT, "include", "dsa.h"), os.path.join(torch, "version.py"), __file__]
    if not force and os.path.exists(BINDING) and \
            all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps):
        return None
    if not shutil.which("g++") or not os.path.exists(os.path.join(python, "Python.h")):
        _drop_binding()
        return None
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"__version__ = '([^']+)'", f.read())
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
            f'-DDSA_STAMP="{binding_stamp(version.group(1) if version else "")}"', *(f"-I{p}" for p in inc), BINDING_SRC, "-o", BINDING + ".tmp", "-L" + os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _build_binding(cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode == 0:
        os.replace(BINDING + ".tmp", BINDING)
    else:
        _drop_binding()
        print("_binding.so not built, Python marshals the serving calls:\n" + r.stderr[-2000:], file=sys.stderr)


def build(verbose: bool = False, force: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _stale(o, s):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            print(" ".join(cmd))
        return cmd

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        cmd = _binding_job(nvcc, force)
        binding = ex.submit(_build_binding, cmd) if cmd else None
        list(ex.map(run, jobs))
        if binding:
            binding.result()
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
