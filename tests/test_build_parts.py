"""What is built needs no more than it uses: the library nvcc alone, the binding the library alone. The module of
csrc/calls.cpp is an addition to both, and one for each torch and Python."""
import os
import subprocess
import sys

import pytest
import torch

from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    moe.load()


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return r


def test_library_is_built_without_torch():
    python(f"""
import runpy, sys
sys.modules["torch"] = None  # importing it fails
b = runpy.run_path({os.path.join(ROOT, "routing_dispatch_expert_gb300", "build.py")!r})
assert b["build"]() == {pkg_build.SO!r} and b["calls_path"]() is None
""")


def test_library_is_loaded_without_the_module():
    """Every call is there; those of the module are made by the steps in Python, which come to the same checks."""
    r = python("""
import torch
from routing_dispatch_expert_gb300 import build, moe
build.calls_path = lambda: build.OUT_DIR + "/none.so"
moe.load()
assert moe.workspace_size(moe.make_config(4, 256, 8, 2, 256)) > 0 and moe.launch_count() == 0
for call in (lambda: moe.rms_norm(torch.zeros(2, 2)), lambda: moe.permute(moe.make_config(2, 256, 8, 2, 256), torch.zeros(2, 2),
             torch.zeros(2, 2), None)):
    try:
        call()
    except ValueError as e:
        assert "must be a CUDA tensor" in str(e)
    else:
        raise AssertionError
""")
    assert "take longer" in r.stderr


def test_a_module_that_cannot_be_made_does_not_stop_the_build(monkeypatch, tmp_path):
    monkeypatch.setattr(pkg_build, "calls_path", lambda: str(tmp_path / "_calls.so"))
    for compile_, link in ((["false"], ["false"]), (["/no/such/compiler"], ["false"])):
        monkeypatch.setattr(pkg_build, "_calls_commands", lambda module: (compile_, link))
        with pytest.warns(UserWarning, match="not compiled"):
            assert pkg_build.build() == pkg_build.SO
    monkeypatch.setattr(pkg_build, "_calls_commands", lambda module: (["touch", str(tmp_path / "_calls.o")], ["false"]))
    with pytest.warns(UserWarning, match="not linked"):
        assert pkg_build.build() == pkg_build.SO


def test_module_is_of_this_torch_and_python():
    path = pkg_build.calls_path()
    assert torch.__version__ in path and sys.implementation.cache_tag in path and os.path.exists(path)
    assert moe._calls.__spec__.origin == path


@pytest.mark.gpu
def test_calls_without_the_module():
    python("""
import torch, warnings
warnings.simplefilter("ignore")
from routing_dispatch_expert_gb300 import build, moe
build.calls_path = lambda: build.OUT_DIR + "/none.so"
x, r = torch.randn(9, 40, device="cuda"), torch.randn(9, 40, device="cuda")
y, total = moe.rms_norm(x, None, r)
assert type(moe._calls) is moe._NoCalls and moe.launch_count() == 1 and torch.equal(total, x + r)
x.requires_grad_()
cfg = moe.make_config(9, 256, 8, 2, 256)
idx, w = moe.route_weights(cfg, torch.randn(9, 8, device="cuda").requires_grad_())
s = moe.sort_tokens(cfg, idx, w.detach())
y = moe.unpermute(cfg, moe.permute(cfg, x, s["inv_pos"], s["offsets"]), s["inv_pos"], w, r, s["offsets"])
y.sum().backward()
want = w.detach().sum(1, keepdim=True).expand_as(x)
assert (x.grad - want).abs().max() < 1e-6
""")
