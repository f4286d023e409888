"""Build libpd.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and the
CPython module between it and torch's tensors (pd_binding.so) with g++.  Without
PyTorch the library alone is built.

Each translation unit compiles in its own nvcc process, in parallel; the
objects and the shared library land in ``paged_kv_decode_splitk_gb300/_build``.
"""

from __future__ import annotations

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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpd.so")
BINDING = os.path.join(BUILD, "pd_binding.so")

SOURCES = ["pd_api.cu", "pd_small.cu", "pd_unit_d64.cu", "pd_unit_d128.cu", "pd_unit_d256.cu",
           "pd_unit_fp8_d64.cu", "pd_unit_fp8_d128.cu", "pd_unit_fp8_d256.cu", "pd_noalloc.cu", "pd_rope.cu",
           "pd_unit_own_d64.cu", "pd_unit_own_d128.cu", "pd_unit_own_d256.cu", "pd_prefix.cu", "pd_prefix_d64.cu",
           "pd_prefix_d128.cu", "pd_prefix_d256.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA translation unit and link libpd.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "pd.h"))
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    # (torch found, not imported: the machine that builds need not load it)
    torch = importlib.util.find_spec("torch")
    if torch is not None:
        torch = torch.submodule_search_locations[0]
        src, obj, version = os.path.join(CSRC, "pd_binding.cpp"), os.path.join(BUILD, "pd_binding.o"), os.path.join(torch, "version.py")
        if force or _stale(obj, [src, os.path.join(INCLUDE, "pd.h"), version]):
            cuda = os.path.dirname(os.path.dirname(shutil.which(nvcc) or nvcc))
            built_for = re.search(r"__version__ = ['\"](.*)['\"]", open(version).read()).group(1)
            cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-fvisibility=hidden", f'-DPD_TORCH_VERSION="{built_for}"', f"-I{INCLUDE}",
                   "-isystem", f"{torch}/include", "-isystem", f"{torch}/include/torch/csrc/api/include", "-isystem", f"{cuda}/include",
                   f"-I{sysconfig.get_paths()['include']}", "-c", src, "-o", obj]
            procs.append(("pd_binding.cpp", subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        msg = "\n".join(f"--- {src}\n{log}" for src, log in failed)
        raise RuntimeError(f"the compiler failed:\n{msg}")
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fvisibility=hidden"]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if torch is not None and (force or _stale(BINDING, [obj, LIB])):
        tmp = BINDING + f".tmp{os.getpid()}"
        libs = [f"-l{name}" for name in ("torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda")]
        subprocess.run(["g++", "-shared", obj, LIB, f"-L{torch}/lib", *libs, "-Wl,-rpath,$ORIGIN", "-o", tmp], check=True)
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
