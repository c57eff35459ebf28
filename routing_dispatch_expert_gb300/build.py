"""Build libmoe_gb300.so in-tree with nvcc for sm_103a (one -gencode, sources compiled in parallel), and, where there is
torch, the Python module of the calls around the experts (csrc/calls.cpp). The library needs nvcc alone; the binding
does without the module, at a longer host time of a call."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
SO = os.path.join(OUT_DIR, "libmoe_gb300.so")
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


def calls_path() -> str | None:
    """The module of csrc/calls.cpp for the torch and Python that run: it uses interfaces of both that change from version to
    version. None without torch."""
    try:
        from torch.version import __version__ as torch_version
    except ImportError:
        return None
    return os.path.join(OUT_DIR, f"_calls.torch-{torch_version}.{sys.implementation.cache_tag}.so")


def _calls_commands(module: str) -> tuple[list[str], list[str]]:
    """Compiler and linker of csrc/calls.cpp."""
    import torch

    top, obj = os.path.dirname(torch.__file__), module[:-3] + ".o"
    include = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *(a for i in include for a in ("-isystem", i)), "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj]
    link = ["g++", "-shared", "-o", module, obj, "-L" + OUT_DIR, "-l:libmoe_gb300.so", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link


def _run(cmd: list[str]) -> tuple[int, str]:
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return 1, str(e)
    return r.returncode, r.stdout + r.stderr


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
    module = calls_path()
    compile_calls, link_calls = _calls_commands(module) if module else (None, None)
    if module and (force or _newer(module[:-3] + ".o", [os.path.join(CSRC, "calls.cpp"), include])):
        jobs.append(compile_calls)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(_run, jobs))
        for cmd, (rc, text) in zip(jobs, results):
            if verbose or (rc != 0 and cmd is not compile_calls):
                print(" ".join(cmd))
                print(text)
            if rc != 0 and cmd is compile_calls:
                module = None
                warnings.warn("csrc/calls.cpp was not compiled, small calls take longer: " + text.strip()[-300:])
            elif rc != 0:
                raise RuntimeError(f"{cmd[0]} failed for {cmd[-3]}")
    if force or _newer(SO, objs):
        subprocess.check_call(["nvcc", *ARCH, "-shared", "-cudart", "shared", "-o", SO, *objs])
    if module and (force or _newer(module, [module[:-3] + ".o", SO])):
        rc, text = _run(link_calls)
        if rc != 0:
            warnings.warn("csrc/calls.cpp was not linked, small calls take longer: " + text.strip()[-300:])
    return SO


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
