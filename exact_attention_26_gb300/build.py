"""Build libfa.so (the CUDA library behind include/fa.h) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel, then linked into
``exact_attention_26_gb300/_lib/libfa.so`` against the shared CUDA runtime.  Beside it,
``_fa_torch.so`` is the CPython extension that makes the paged-cache calls on torch tensors
(host code only, compiled against the installed torch's headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libfa.so")
EXT = os.path.join(OUT_DIR, "_fa_torch.so")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_decode.cu", "fa_noalloc.cu", "fa_quant.cu",
           "fa_probe.cu", "fa_cache.cu", "fa_decode_fp8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")


def compile_flags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-I", INCLUDE, "-I", CSRC, *extra]


def _torch_flags():
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    lib = os.path.join(root, "lib")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    compile_ = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
                "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda_inc]
    link = ["-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    return compile_, link


def _compile_ext(obj_dir):
    """Object file of the torch front end (linked once libfa.so exists)."""
    obj = os.path.join(obj_dir, "fa_torch.o")
    cmd = ["g++", *_torch_flags()[0], "-c", os.path.join(CSRC, "fa_torch.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for fa_torch.cpp:\n{' '.join(cmd)}\n{res.stderr}")
    return obj


def _link_ext(obj):
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", *_torch_flags()[1]]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stderr}")
    os.replace(tmp, EXT)


def build(verbose: bool = False, extra_flags=(), ptxas_info: bool = False) -> str:
    nvcc = _nvcc()
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    flags = compile_flags(extra_flags)
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def one(src):
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{res.stderr}")
        return obj, res.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_compile_ext, obj_dir)
        results = list(ex.map(one, SOURCES))
        ext_obj = ext.result()
    if verbose or ptxas_info:
        for (_, log), src in zip(results, SOURCES):
            if log.strip():
                print(f"--- {src}\n{log}")
    tmp = LIB + f".tmp{os.getpid()}"
    libdir = _cuda_lib_dir(nvcc)
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *[o for o, _ in results],
           "-Xlinker", f"-rpath,{libdir}", "-Xlinker", "-soname,libfa.so"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stderr}")
    os.replace(tmp, LIB)
    _link_ext(ext_obj)
    return LIB


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            if os.path.getmtime(os.path.join(d, f)) > t:
                return True
    return False


if __name__ == "__main__":
    import sys
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
