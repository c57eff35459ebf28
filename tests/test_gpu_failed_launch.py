"""A launch that fails on the host is reported at once: the call is not made a second time. The failure is that of a stream
whose capture another call has ended: every launch there returns an error, and none reaches the GPU."""
import contextlib
import ctypes

import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe

pytestmark = pytest.mark.gpu
RELAXED, UNSUPPORTED, INVALIDATED = 2, 900, 901


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


@contextlib.contextmanager
def ended_capture(stream):
    """Within, every launch on the stream fails on the host."""
    rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    s = ctypes.c_void_p(stream.cuda_stream)
    assert rt.cudaStreamBeginCapture(s, RELAXED) == 0
    assert rt.cudaStreamSynchronize(s) == UNSUPPORTED  # not allowed in a capture, and the end of it
    rt.cudaGetLastError()
    try:
        yield
    finally:
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) == INVALIDATED and not graph.value
        rt.cudaGetLastError()


def calls():
    """One launch each, and two."""
    x, w = torch.randn(64, 256, device="cuda"), torch.ones(256, device="cuda")
    cfg = rde.make_config(T=5000, h=256, E=64, k=2, I=256)
    idx = torch.randint(0, 64, (5000, 2), device="cuda", dtype=torch.int32)
    s = rde.sort_tokens(cfg, idx)
    rows, yd = torch.randn(5000, 64, device="cuda"), torch.randn(10000, 64, device="cuda")
    tw, z = torch.ones(5000, 2, device="cuda"), torch.randn(5000, 64, device="cuda")
    return {"rms_norm": lambda: rde.rms_norm(x, w), "rms_norm_backward": lambda: rde.rms_norm_backward(x, x, w),
            "sort_tokens": lambda: rde.sort_tokens(cfg, idx), "permute": lambda: rde.permute(cfg, rows, s["inv_pos"], s["offsets"]),
            "unpermute": lambda: rde.unpermute(cfg, yd, s["inv_pos"]),
            "unpermute_backward": lambda: rde.unpermute_backward(cfg, rows, yd, s["inv_pos"], s["offsets"]),
            "route_backward": lambda: rde.route_backward(cfg, z, idx, tw)}


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_backward", "sort_tokens", "permute", "unpermute", "unpermute_backward",
                                  "route_backward"])
def test_reported_at_once(monkeypatch, name):
    call, stream = calls()[name], torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call()  # the outputs' memory is the stream's from here on
        stream.synchronize()
        steps = []
        monkeypatch.setattr(moe, "_plain", lambda *a: steps.append(name))
        before = rde.launch_count()
        with ended_capture(stream), pytest.raises(rde.MoeError, match="launch") as e:
            call()
        assert e.value.code == moe.MOE_ERR_CUDA and rde.launch_count() == before
        assert not steps  # those of the binding, which would make the call again
        monkeypatch.undo()
        call()
        stream.synchronize()


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_backward", "sort_tokens", "permute", "unpermute", "unpermute_backward",
                                  "route_backward"])
def test_nothing_is_left_behind(name):
    """The error is the call's alone: the runtime's last error, which the next launch of any other code looks at, is clear."""
    call, stream = calls()[name], torch.cuda.Stream()
    rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call()
        stream.synchronize()
        with ended_capture(stream):
            with pytest.raises(rde.MoeError):
                call()
            assert rt.cudaPeekAtLastError() == 0
