"""Builds librope_chain.so in-tree with nvcc for sm_103a, and the Python
module _draft.so (csrc/py_draft.cpp: the drafted tokens' calls) with g++.

Each .cu under csrc/ and the module's source compile to an object in parallel,
then the shared library and the module are linked next to this file.  ptxas
register/spill reports are kept in _build/ptxas.log.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "librope_chain.so")
MODULE = os.path.join(HERE, "_draft.so")
SOURCES = ["rc_api.cu", "k1_norms.cu", "k2_gemm.cu", "k3_store.cu", "k4_qkv_front.cu",
           "rc_project_static.cu", "k5_tree_attention.cu", "k6_rope.cu", "k7_logits.cu", "rc_draft.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# --fmad=false: no multiply-add is fused unless the source asks for it.
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--fmad=false", "-Xcompiler", "-fPIC",
                "-Xcompiler", "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"),
                 os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"),
                 shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or CUDA_HOME)")


def _torch_flags():
    """Compiler and linker flags of a module that uses torch's C++ tensors."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    lib = os.path.join(root, "lib")
    compile_flags = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I", include,
                     "-I", os.path.join(include, "torch", "csrc", "api", "include"),
                     "-I", sysconfig.get_paths()["include"], "-I", cuda,
                     "-I", os.path.join(ROOT, "include"),
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    link_flags = ["-L" + lib, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda",
                  "-Wl,-rpath," + lib, "-Wl,-rpath,$ORIGIN"]
    return compile_flags, link_flags


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(ROOT, "include", "rope_chain.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr + r.stdout

    cxx = shutil.which("g++") or "c++"
    compile_flags, link_flags = _torch_flags()

    def compile_module():
        obj = os.path.join(BUILD, "py_draft.o")
        cmd = [cxx, *compile_flags, "-c", os.path.join(CSRC, "py_draft.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on py_draft.cpp:\n{r.stdout}\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        module = ex.submit(compile_module)
        results = list(ex.map(compile_one, SOURCES))
        module_obj = module.result()
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for _, log in results:
            f.write(log)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = MODULE + f".{os.getpid()}.tmp"
    cmd = [cxx, "-shared", "-o", tmp, module_obj, "-L" + HERE, "-lrope_chain", *link_flags]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the module failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MODULE)
    if verbose:
        print(open(os.path.join(BUILD, "ptxas.log")).read())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
