"""Builds libmsa.so in-tree from csrc/*.cu for sm_103a (nvcc, no cmake), and the
native part of the Python binding, _msa_torch.so, from csrc/binding.cpp (g++).

Objects go to msa_block_sparse_gb300/_build/, the libraries to
msa_block_sparse_gb300/.  Translation units compile in parallel; a unit is rebuilt
when it or any header is newer than its object.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmsa.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_msa_torch.so")
GENCODE = "arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _flags():
    return ["-gencode", GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
            "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "msa.h"))
    return hs


def _compile(src: str, obj: str, verbose: bool):
    cmd = [nvcc(), *_flags(), "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
    return r.stderr


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _compile_binding(obj: str):
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-I", sysconfig.get_paths()["include"], "-c", BINDING_SRC, "-o", obj], "g++ for binding.cpp")


def _link_binding(obj: str):
    import torch
    tmp = BINDING + ".tmp"
    _run([shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-lmsa",
          "-Wl,-rpath,$ORIGIN", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"], "link of the binding")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdr_time = max(os.path.getmtime(h) for h in _headers())
    jobs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        stale = force or not os.path.exists(obj) or \
            os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time)
        jobs.append((src, obj, stale))
    logs = []
    bobj = os.path.join(BUILD, "binding.o")
    bstale = force or not os.path.exists(bobj) or os.path.getmtime(bobj) < max(
        os.path.getmtime(BINDING_SRC), os.path.getmtime(os.path.join(ROOT, "include", "msa.h")))
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        bfut = ex.submit(_compile_binding, bobj) if bstale else None
        futs = {ex.submit(_compile, s, o, verbose): s for s, o, st in jobs if st}
        for f in cf.as_completed(futs):
            logs.append(f.result())
        if bfut:
            bfut.result()
    objs = [o for _, o, _ in jobs]
    if force or any(st for _, _, st in jobs) or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), "-gencode", GENCODE, "-shared", "-cudart", "shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if bstale or not os.path.exists(BINDING):
        _link_binding(bobj)
    if verbose:
        sys.stderr.write("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
