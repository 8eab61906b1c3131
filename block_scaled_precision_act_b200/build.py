"""Build ``libbsp.so`` in-tree with nvcc for sm_100a (B200), and ``_fastcall.so``, the binding's
C++ short cut, with g++ against the installed torch.

No fast-math and no flush-to-zero: the quantizers rely on IEEE division,
reciprocal and denormals to produce codes bit-identical to their definition.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbsp.so")
FASTCALL = os.path.join(PKG, "_fastcall.so")
SOURCES = ["api_common.cu", "quant.cu", "gemm.cu", "linear.cu", "linear_noalloc.cu", "gemv.cu",
           "gemv_direct.cu", "fp8kv_append.cu", "fp8kv_attention.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _flags(verbose_ptxas: bool):
    f = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _deps():
    hdrs = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    hdrs += [os.path.join(INCLUDE, h) for h in os.listdir(INCLUDE)]
    return max(os.path.getmtime(p) for p in hdrs)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdr_time = _deps()
    objs = []
    jobs = []
    for src in SOURCES:
        sp = os.path.join(CSRC, src)
        op = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(op)
        if (force or verbose_ptxas or not os.path.exists(op)
                or os.path.getmtime(op) < max(os.path.getmtime(sp), hdr_time)):
            jobs.append([NVCC] + _flags(verbose_ptxas) + ["-c", sp, "-o", op])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        for out in ex.map(run, jobs):
            if verbose_ptxas and out:
                print(out)
    if (jobs or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        tmp = LIB + f".tmp{os.getpid()}"
        run([NVCC] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    build_fastcall(run, force)
    return LIB


def build_fastcall(run, force: bool) -> None:
    src = os.path.join(CSRC, "fastcall.cpp")
    if (not force and os.path.exists(FASTCALL)
            and os.path.getmtime(FASTCALL) >= max(os.path.getmtime(src), _deps())):
        return
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = cpp_extension.include_paths(device_type="cuda") + [sysconfig.get_paths()["include"],
                                                             INCLUDE]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = FASTCALL + f".tmp{os.getpid()}"
    run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wextra",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         *[x for d in inc for x in ("-isystem", d)], src, "-o", tmp, "-L", libs, "-lc10",
         "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-L", PKG, "-l:libbsp.so",
         "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, FASTCALL)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
