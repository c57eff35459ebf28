"""The calls of csrc/calls.cpp against the same steps in Python: the same outputs, in shape, type and bits; which calls it
takes; and what becomes of those that it does not."""
import gc
import threading

import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe

pytestmark = pytest.mark.gpu
F32, BF16, F16, U8 = torch.float32, torch.bfloat16, torch.float16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


class Counting:
    """The native calls, counted; `declines`: none of them is taken."""

    def __init__(self, calls, declines):
        self.calls, self.declines, self.taken = calls, declines, 0

    def __getattr__(self, name):
        def call(*a):
            out = None if self.declines else getattr(self.calls, name)(*a)
            self.taken += out is not None
            return out
        return call


def both_ways(monkeypatch, f):
    native, got = moe._calls, []
    for declines in (False, True):
        counting = Counting(native, declines)
        monkeypatch.setattr(moe, "_calls", counting)
        got.append((f(), counting.taken))
    monkeypatch.setattr(moe, "_calls", native)
    (a, n), (b, none) = got
    assert n == 1 and none == 0
    flat = lambda v: list(v.values()) if isinstance(v, dict) else list(v) if isinstance(v, tuple) else [v]  # noqa: E731
    assert type(a) is type(b) and (not isinstance(a, dict) or list(a) == list(b)) and len(flat(a)) == len(flat(b))
    for p, q in zip(flat(a), flat(b)):
        assert (p is None) == (q is None)
        if p is not None:
            assert p.dtype == q.dtype and p.shape == q.shape and p.stride() == q.stride() and p.device == q.device
            assert torch.equal(p.view(U8) if p.dtype == U8 else p, q)
    return a


@pytest.mark.parametrize("kind", [F32, BF16, F16])
@pytest.mark.parametrize("rows", [0, 1, 5])
def test_norm(monkeypatch, kind, rows):
    for cols, ld in ((64, 64), (65, 70), (1, 1), (1, 9)):
        x = torch.randn(rows, ld, device="cuda").to(kind)[:, :cols]
        for other in (None, kind, F32):
            r = None if other is None else torch.randn(rows, ld, device="cuda").to(other)[:, :cols]
            for w in (None, torch.ones(cols, device="cuda"), torch.ones(cols, device="cuda").to(kind)):
                both_ways(monkeypatch, lambda: rde.rms_norm(x, w, r, 1e-5))
                both_ways(monkeypatch, lambda: rde.rms_norm_fp8(x, w, r))
                both_ways(monkeypatch, lambda: rde.rms_norm_fp8(x, w, r, with_y=True))
                dy = torch.randn(rows, cols, device="cuda").to(kind)
                t = x if r is None else r
                dt = torch.randn(rows, cols, device="cuda").to(t.dtype)
                dx, dr, dw = both_ways(monkeypatch, lambda: rde.rms_norm_backward(dy, t, w, 1e-5, dt))
                assert (dr is dx) == (t.dtype == kind) and (dw is None) == (w is None)
                both_ways(monkeypatch, lambda: rde.rms_norm_backward(dy, t, w, weight_gradient=False))
                ws = rde.rms_norm_backward_workspace(rows, cols)
                both_ways(monkeypatch, lambda: rde.rms_norm_backward(dy, t, w, 1, None, True, ws))


@pytest.mark.parametrize("T,E,k", [(0, 4, 2), (1, 4, 2), (700, 16, 4)])
def test_rows(monkeypatch, T, E, k):
    cfg = rde.make_config(T=T, h=256, E=E, k=k, I=256, capacity_factor=1.5)
    idx = torch.randint(-1, E, (T, k), device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, device="cuda")
    both_ways(monkeypatch, lambda: rde.sort_tokens(cfg, idx))
    both_ways(monkeypatch, lambda: rde.sort_tokens(cfg, idx, w, rde.sort_tokens_workspace(cfg)))
    s = both_ways(monkeypatch, lambda: rde.sort_tokens(cfg, idx, w))
    for kind in (F32, BF16, F16, U8):
        x = torch.randn(T, 72, device="cuda").to(kind)[:, :65]
        both_ways(monkeypatch, lambda: rde.permute(cfg, x, s["inv_pos"], s["offsets"]))
        if kind is U8:
            scales = torch.rand(T, 1, device="cuda")
            both_ways(monkeypatch, lambda: rde.permute(cfg, x, s["inv_pos"], s["offsets"], scales))
            continue
        yd, base, dy = (torch.randn(n, 65, device="cuda").to(kind) for n in (T * k, T, T))
        for v in (None, w):
            for b in (None, base):
                both_ways(monkeypatch, lambda: rde.unpermute(cfg, yd, s["inv_pos"], v, b))
            for rows in (None, yd):
                both_ways(monkeypatch, lambda: rde.unpermute_backward(cfg, dy, rows, s["inv_pos"], s["offsets"], v))
    for kind in (F32, BF16):
        both_ways(monkeypatch, lambda: rde.route_backward(cfg, torch.randn(T, E, device="cuda").to(kind) * 0 + 0.5, idx, w))


def test_under_a_placement(monkeypatch):
    import numpy as np

    plan = rde.eplb_plan(np.arange(8) + 1, 4, 4)
    cfg = rde.make_config(T=300, h=256, E=8, k=2, I=256, placement=rde.Placement(plan))
    idx = torch.randint(0, 8, (300, 2), device="cuda", dtype=torch.int32)
    s = both_ways(monkeypatch, lambda: rde.sort_tokens(cfg, idx))
    assert s["counts"].numel() == plan["slot_expert"].size and int(s["offsets"][-1]) == 600
    both_ways(monkeypatch, lambda: rde.permute(cfg, torch.ones(300, 64, device="cuda"), s["inv_pos"], s["offsets"]))


def test_what_is_not_taken_is_refused_in_words():
    """None of these launches anything; each says what is wrong, as the checks in Python do."""
    cfg = rde.make_config(T=4, h=256, E=8, k=2, I=256)
    x, idx = torch.randn(4, 64, device="cuda"), torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    off = torch.zeros(9, device="cuda", dtype=torch.int32)
    before = rde.launch_count()
    for call, words in (
            (lambda: rde.rms_norm(x.double()), "x must be"), (lambda: rde.rms_norm(x.cpu()), "x must be a CUDA tensor"),
            (lambda: rde.rms_norm(x.t()), "contiguous"), (lambda: rde.rms_norm(x, x[0, :63]), "weight"),
            (lambda: rde.rms_norm(x, None, x[:3]), "residual"), (lambda: rde.rms_norm(x[0]), "x must"),
            (lambda: rde.rms_norm_backward(x[:, :60], x), "dy"), (lambda: rde.rms_norm_backward(x, x.half()), "total"),
            (lambda: rde.sort_tokens(cfg, idx.long()), "topk_idx"), (lambda: rde.sort_tokens(cfg, idx, idx), "topk_w"),
            (lambda: rde.permute(cfg, x[:3], idx, off), "x must"), (lambda: rde.permute(cfg, x, idx, off[:8]), "offsets"),
            (lambda: rde.permute(cfg, x, idx, off, x), "x must"), (lambda: rde.unpermute(cfg, x, idx), "yd"),
            (lambda: rde.unpermute_backward(cfg, x, x, idx, off), "yd"), (lambda: rde.route_backward(cfg, x, idx, x), "logits")):
        with pytest.raises(ValueError, match=words):
            call()
    with pytest.raises(rde.MoeError, match="eps"):
        rde.rms_norm(x, eps=-1.0)
    with pytest.raises(rde.MoeError, match="16-byte"):
        rde.rms_norm(torch.randn(300, device="cuda")[1:65].view(1, 64))
    with pytest.raises(rde.MoeError, match="too small"):
        rde.rms_norm_backward(x, x, x[0].contiguous(), ws=torch.empty(16, device="cuda", dtype=U8))
    for bad in (None, 3, b"0" * 64, rde.make_config):
        with pytest.raises((AttributeError, TypeError, ctypes_error())):
            rde.sort_tokens(bad, idx)
    assert rde.launch_count() == before


def ctypes_error():
    import ctypes

    return ctypes.ArgumentError


def test_nothing_is_kept():
    """Outputs go when their names do, and inputs are not held: the memory in use is the same after many calls."""
    cfg = rde.make_config(T=64, h=256, E=8, k=2, I=256)
    x, idx, w = torch.randn(64, 256, device="cuda"), torch.randint(0, 8, (64, 2), device="cuda", dtype=torch.int32), torch.rand(64, 2, device="cuda")

    def once():
        s = rde.sort_tokens(cfg, idx, w)
        xd = rde.permute(cfg, x, s["inv_pos"], s["offsets"])
        y, t = rde.rms_norm(rde.unpermute(cfg, xd, s["inv_pos"], w, x), x[0], x)
        rde.rms_norm_backward(y, t, x[0], 1e-6)
        rde.unpermute_backward(cfg, y, xd, s["inv_pos"], s["offsets"], w)
        for bad in (x.cpu(), x.double()):
            with pytest.raises(ValueError):
                rde.rms_norm(bad)

    once()
    gc.collect()
    used = torch.cuda.memory_allocated()
    for _ in range(200):
        once()
    gc.collect()
    assert torch.cuda.memory_allocated() == used


def test_from_threads_on_streams():
    x = torch.randn(64, 1024, device="cuda").to(BF16)
    want, wrong = rde.rms_norm(x), []
    torch.cuda.synchronize()

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                if not torch.equal(rde.rms_norm(x), want):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
