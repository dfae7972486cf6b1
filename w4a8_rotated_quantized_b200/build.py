"""Build the in-tree CUDA library (sm_100a only) with nvcc, and the extension module ``_calls`` with g++.

The shared library is written next to this file as ``libconvrot_b200.so``
and object files go to ``_build/``.  nvcc cross-compiles for sm_100a on a
machine without a GPU.  ``_calls.so`` marshals the calls whose GPU time is a
few microseconds; it is compiled against the installed torch and links to the
library beside it.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libconvrot_b200.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "py_calls.cpp")
CALLS_MADE_WITH = os.path.join(BUILD, "_calls.made_with")
SOURCES = ["api.cu", "act_kernels.cu", "gemm_w4a4.cu", "gemm_w4a4_pair.cu", "gemm_w4a4_small.cu", "gemm_i8.cu",
           "gemm_w4a8.cu", "gemm_a8w4.cu", "tmap.cu", "noalloc.cu",
           "selftest.cu", "api_adapters.cu", "lora_rows.cu", "lora_mma.cu", "grad_values.cu", "ckpt_mma.cu", "gemm_bf16.cu",
           "grad_input_few.cu"]
HEADERS = [os.path.join(ROOT, "include", "convrot.h")] + [
    os.path.join(CSRC, f) for f in ("cr_device.cuh", "cr_internal.h", "act_device.cuh", "grid_sync.cuh", "lora_device.cuh",
                                    "unit_device.cuh", "lost_wait.cuh", "f16_device.cuh")
]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=default",
         f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _mtime(p: str) -> float:
    return os.path.getmtime(p) if os.path.exists(p) else -1.0


def _calls_cmd() -> list:
    import torch

    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(t, "include"),
            "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"), "-isystem", cuda, CALLS_SRC,
            "-o", CALLS, "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(t, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _calls_made_with() -> str:
    """What _calls.so is bound to beside its own source: this Python and the torch that it is compiled against."""
    torch = importlib.util.find_spec("torch")
    return "\n".join([sys.version, importlib.metadata.version("torch"), torch.origin if torch else ""])


def _calls_stale() -> bool:
    if _mtime(CALLS) < max(_mtime(CALLS_SRC), _mtime(HEADERS[0])) or not os.path.exists(CALLS_MADE_WITH):
        return True
    with open(CALLS_MADE_WITH) as f:
        return f.read() != _calls_made_with()


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every .cu source and link the shared library; return its path."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdr_time = max(_mtime(h) for h in HEADERS)
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or ptxas_info or _mtime(o) < max(_mtime(s), hdr_time):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        for err in ex.map(run, jobs):
            if verbose and err:
                sys.stderr.write(err)
    if jobs or force or _mtime(LIB) < max(_mtime(o) for o in objs):
        run([nvcc, *ARCH, "-shared", "-o", LIB, *objs])
    if force or _calls_stale():
        run(_calls_cmd())
        with open(CALLS_MADE_WITH, "w") as f:
            f.write(_calls_made_with())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
