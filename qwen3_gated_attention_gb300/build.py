"""Build libgattn.so (sm_103a) in-tree with nvcc, one process per translation unit, and,
where torch is found, the module _paged beside it (tensor arguments of the paged-cache calls).

Usage: ``python -m qwen3_gated_attention_gb300.build [--force] [--verbose-ptxas]``
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
# the packed-sequence operators (prompt pass, delta rule)
CSRC_SEQ = os.path.join(PKG, "csrc_seq")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgattn.so")
# host code that reads torch tensors
TENSORS = os.path.join(PKG, "csrc_torch", "paged_tensors.cpp")
MODULE = os.path.join(PKG, "_paged.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return [os.path.join(d, f) for d in (CSRC, CSRC_SEQ) for f in sorted(os.listdir(d))
            if f.endswith((".cu", ".cpp"))]


def _headers():
    hs = [os.path.join(d, f) for d in (CSRC, CSRC_SEQ) for f in os.listdir(d)
          if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "gattn.h"))
    return hs


def _compile(src, nvcc, verbose_ptxas):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest_dep = max(os.path.getmtime(p) for p in _headers() + [src, __file__])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj, None
    cmd = [nvcc, "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
           "-I", CSRC, "-I", CSRC_SEQ, "-c", src, "-o", obj + ".tmp"]
    if src.endswith(".cpp"):
        cmd = [nvcc, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-c", src, "-o",
               obj + ".tmp"]
    elif verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return obj, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    os.replace(obj + ".tmp", obj)
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj, None


def has_torch():
    """Whether there is a torch to build the tensor module against."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _compile_module(src):
    """The object of the tensor module (C++ against torch's headers, no CUDA); None without
    torch."""
    import sysconfig

    if not has_torch():
        return None, None
    import torch
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    dep = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "gattn.h"), __file__,
                                            torch.__file__))
    if os.path.exists(obj) and os.path.getmtime(obj) >= dep:
        return obj, None
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE, "-I",
           inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I",
           sysconfig.get_paths()["include"], "-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return obj, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    os.replace(obj + ".tmp", obj)
    return obj, None


def _link_module(obj):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + ".tmp%d" % os.getpid()
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgattn.so", "-L",
           lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MODULE)


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    if force:
        for s in srcs + [TENSORS]:
            o = os.path.join(BUILD, os.path.basename(s) + ".o")
            if os.path.exists(o):
                os.remove(o)
    with ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        tensors = ex.submit(_compile_module, TENSORS)
        results = list(ex.map(lambda s: _compile(s, nvcc, verbose_ptxas), srcs))
    errors = [e for _, e in results if e]
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    objs = [o for o, _ in results]
    if (not os.path.exists(LIB) or force or
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc, "-shared", *ARCH, "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    # the library stands by now, whatever becomes of the module
    module, error = tensors.result()
    if error:
        raise RuntimeError("tensor module: " + error)
    if module and (not os.path.exists(MODULE) or force or
            os.path.getmtime(MODULE) < max(os.path.getmtime(LIB), os.path.getmtime(module))):
        _link_module(module)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(args.force, args.verbose_ptxas))
