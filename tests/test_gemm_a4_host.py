"""The 4-bit GEMM's launch arithmetic (csrc/gemm_a4_host.h), compiled with g++ and run. No GPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routing_dispatch_expert_gb300", "csrc")


def test_tiles_of_a_launch(tmp_path):
    exe = tmp_path / "gemm_a4_host_check"
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(ROOT, "tests", "gemm_a4_host_check.cpp"),
                           "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.strip() == "ok"
