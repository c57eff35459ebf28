"""Build libmoe_gb300.so in-tree with nvcc for sm_103a (one -gencode, sources compiled in parallel)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
SO = os.path.join(OUT_DIR, "libmoe_gb300.so")
CALLS = os.path.join(OUT_DIR, "_calls.so")  # Python module: tensors' checks and outputs around the library's calls
SOURCES = ["api.cu", "route.cu", "dispatch.cu", "gemm.cu", "gemm_pair.cu", "gemm_fp8.cu", "gemm_fp4.cu", "combine.cu", "eplb.cu", "fused.cu",
           "fp4_quant.cu", "gemm_a4.cu", "balance_loss.cu", "rms_norm.cu", "rms_norm_backward.cu", "permute.cu", "unpermute.cu",
           "route_backward.cu"]
HEADERS = ["common.cuh", "gemm_common.cuh", "kernels.h", "device_state.h", "route_impl.cuh", "dispatch_impl.cuh", "fp4_impl.cuh", "rows.cuh",
           "rms_norm.cuh", "gemm_a4_host.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def _newer(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _calls_commands(obj: str) -> tuple[list[str], list[str]]:
    """Compiler and linker of csrc/calls.cpp."""
    import torch

    top = os.path.dirname(torch.__file__)
    include = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *(a for i in include for a in ("-isystem", i)), "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj]
    link = ["g++", "-shared", "-o", CALLS, obj, "-L" + OUT_DIR, "-l:libmoe_gb300.so", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    include = os.path.join(os.path.dirname(PKG), "include", "moe.h")
    common = [os.path.join(CSRC, h) for h in HEADERS] + [include]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _newer(o, [s] + common):
            jobs.append(["nvcc", *FLAGS, *ARCH, "-c", s, "-o", o])
    calls_obj = os.path.join(OUT_DIR, "calls.o")
    compile_calls, link_calls = _calls_commands(calls_obj)
    if force or _newer(calls_obj, [os.path.join(CSRC, "calls.cpp"), include]):
        jobs.append(compile_calls)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                print(" ".join(cmd))
                print(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"{cmd[0]} failed for {cmd[-3]}")
    if force or _newer(SO, objs):
        subprocess.check_call(["nvcc", *ARCH, "-shared", "-cudart", "shared", "-o", SO, *objs])
    if force or _newer(CALLS, [calls_obj, SO]):
        subprocess.check_call(link_calls)
    return SO


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True))
