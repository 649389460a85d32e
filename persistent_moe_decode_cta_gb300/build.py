"""Build libmk.so (the C-ABI megakernel library) in-tree with nvcc for sm_103a.

Four builds of the megakernel (default, deterministic, two tensor-core variants), the
multi-token operators and the host planner/ABI compile in parallel, then link into
persistent_moe_decode_cta_gb300/libmk.so with the CUDA runtime linked statically.  Beside it,
_ops.so is the Python module that checks and marshals tensors for the operators (against the
installed torch, and left out where there is none; it finds libmk.so by its own directory).  Usable as `python -m persistent_moe_decode_cta_gb300.build`.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmk.so")
MODULE = os.path.join(PKG, "_ops.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["mk_kernel.cu", "mk_kernel_det.cu", "mk_kernel_umma.cu", "mk_kernel_umma_ffn.cu",
           "mk_tree_attention.cu", "mk_experts.cu", "mk_qk_rope.cu", "mk_cache_pages.cu", "mk_ops.cpp", "mk_host.cpp"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra_ptxas=False):
    f = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-maxrregcount=224",
         "-I" + os.path.join(ROOT, "include"), "-I" + CSRC] + ARCH
    if extra_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _module_command(out: str, obj: bool):
    """g++ for the Python module: its object, or the link of it."""
    import sysconfig
    import torch
    home = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    if obj:
        inc = [os.path.join(home, "include"), sysconfig.get_paths()["include"], "/usr/local/cuda/include", os.path.join(ROOT, "include")]
        abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
        return [cxx, "-O2", "-std=c++17", "-fPIC", abi, *["-I" + i for i in inc], "-c", os.path.join(CSRC, "ops_module.cpp"), "-o", out]
    return [cxx, "-shared", "-o", out, os.path.join(OUT_DIR, "ops_module.cpp.o"), "-L" + PKG, "-l:libmk.so", "-L" + os.path.join(home, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    nvcc = nvcc_path()
    os.makedirs(OUT_DIR, exist_ok=True)
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(OUT_DIR, src + ".o")
        lang = ["-x", "cu"] if src.endswith(".cu") else ["-x", "c++"]
        cmds.append([nvcc, *lang, *_flags(ptxas_info and src.endswith(".cu")), "-c",
                     os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)

    with_module = importlib.util.find_spec("torch") is not None

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    def module_object():
        return run(_module_command(os.path.join(OUT_DIR, "ops_module.cpp.o"), True))

    with ThreadPoolExecutor(len(cmds) + 1) as ex:
        module = ex.submit(module_object) if with_module else None
        results = list(ex.map(run, cmds))
    for cmd, r in results:
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    link = [nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs, "-cudart", "static"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(link) + "\n" + r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    # (the library is in place whatever becomes of the module)
    if not with_module:
        sys.stderr.write("torch is not installed: _ops.so, which ops.py needs, is left out\n")
        return LIB
    cmd, r = module.result()
    if r.returncode == 0:
        cmd, r = run(_module_command(MODULE + ".tmp", False))
    if r.returncode != 0:
        raise RuntimeError("the Python module failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(MODULE + ".tmp", MODULE)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
