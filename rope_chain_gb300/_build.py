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
MODULE_SOURCE = "py_draft.cpp"
MODULE_STAMP = os.path.join(BUILD, "module.txt")      # the torch and Python that MODULE was made for
HEADER = os.path.join(ROOT, "include", "rope_chain.h")
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
    # (the version: a torch put in place of another of the same path)
    compile_flags = [f'-DRC_TORCH_VERSION="{torch.__version__}"', "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", include,
                     "-I", os.path.join(include, "torch", "csrc", "api", "include"),
                     "-I", sysconfig.get_paths()["include"], "-I", cuda,
                     "-I", os.path.join(ROOT, "include"),
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    link_flags = ["-L" + lib, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda",
                  "-Wl,-rpath," + lib, "-Wl,-rpath,$ORIGIN"]
    return compile_flags, link_flags


def _run(cmd, what: str) -> str:
    """Runs a compiler; what it printed, or RuntimeError."""
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr + r.stdout


def _link(cmd, target: str) -> None:
    """Links `target` beside its place, then moves it there."""
    tmp = f"{target}.{os.getpid()}.tmp"
    _run([*cmd, "-o", tmp], f"link of {os.path.basename(target)}")
    os.replace(tmp, target)


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _library_stale() -> bool:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != MODULE_SOURCE]
    return _older(LIB, deps + [HEADER, os.path.abspath(__file__)])


def _module_stale(made_for: str) -> bool:
    if _older(MODULE, [os.path.join(CSRC, MODULE_SOURCE), HEADER, os.path.abspath(__file__)]):
        return True
    try:
        with open(MODULE_STAMP) as f:
            return f.read() != made_for
    except OSError:
        return True


def _build_library() -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        return obj, _run([cc, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc on {src}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for _, log in results:
            f.write(log)
    _link([cc, *ARCH, "-shared", *(o for o, _ in results)], LIB)


def _compile_module(compile_flags) -> str:
    obj = os.path.join(BUILD, MODULE_SOURCE.replace(".cpp", ".o"))
    cxx = shutil.which("g++") or "c++"
    _run([cxx, *compile_flags, "-c", os.path.join(CSRC, MODULE_SOURCE), "-o", obj], f"g++ on {MODULE_SOURCE}")
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is missing or older than its sources.  The library wants
    nothing of torch and is in place before a failure of the module is raised."""
    os.makedirs(BUILD, exist_ok=True)

    def module_object():
        """(object or None, linker flags, what it was made for)."""
        compile_flags, link_flags = _torch_flags()
        made_for = " ".join(compile_flags + link_flags)
        if not force and not _module_stale(made_for):
            return None, link_flags, made_for
        return _compile_module(compile_flags), link_flags, made_for

    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(module_object)
        if force or _library_stale():
            _build_library()
    obj, link_flags, made_for = module.result()
    if obj is not None:
        _link([shutil.which("g++") or "c++", "-shared", obj, "-L" + os.path.dirname(LIB), "-lrope_chain", *link_flags],
              MODULE)
        with open(MODULE_STAMP, "w") as f:
            f.write(made_for)
    if verbose:
        print(open(os.path.join(BUILD, "ptxas.log")).read())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
