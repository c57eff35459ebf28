"""The norm, sort, permutation and routing gradient without a GPU: refusals (each returns before any CUDA call),
workspace sizes, the binding's checks, and the 64-bit definitions that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import plain_rows as plain
from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe

P = ctypes.c_void_p(0x1000)  # aligned, never read: the calls fail before
ODD = ctypes.c_void_p(0x1008)
BIG = ctypes.c_size_t(1 << 40)


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return moe.load()


def _cfg(**kw):
    return moe.make_config(**{**dict(T=64, h=256, E=8, k=2, I=256), **kw})


def _refused(lib, got, code, text):
    assert got == code, lib.moe_last_error()
    assert text in lib.moe_last_error().decode()


@pytest.mark.parametrize("change,code,text", [
    (dict(rows=-1), -1, "rows must be"), (dict(cols=0), -1, "cols positive"), (dict(cols=16385), -2, "16384"),
    (dict(rows=1 << 31), -2, "int32"), (dict(type=3), -1, "element type"), (dict(rtype=2), -1, "residual must be"),
    (dict(wtype=2), -1, "weight must be"), (dict(eps=-1.0), -1, "eps"), (dict(eps=math.nan), -1, "eps"),
    (dict(s=None), -1, "go together"), (dict(y=None, q=None, s=None), -1, "neither"), (dict(r=None), -1, "total is x"),
    (dict(ldx=63), -1, "ldx"), (dict(ldr=63), -1, "ldr"), (dict(x=None), -1, "x is NULL"), (dict(x=ODD), -1, "x must be"),
    (dict(r=ODD), -1, "residual must be 16"), (dict(w=ODD), -1, "weight must be 16"), (dict(y=ODD), -1, "y must be"),
    (dict(total=ODD), -1, "total must be"), (dict(q=ODD), -1, "q must be"), (dict(s=ODD), -1, "s must be"),
])
def test_norm_refusals(lib, change, code, text):
    a = {**dict(x=P, type=1, rows=4, cols=64, ldx=64, r=P, rtype=1, ldr=64, w=P, wtype=0, eps=1e-6, y=P, total=P, q=P, s=P),
         **change}
    _refused(lib, lib.moe_rms_norm(a["x"], a["type"], a["rows"], a["cols"], a["ldx"], a["r"], a["rtype"], a["ldr"], a["w"],
                                   a["wtype"], a["eps"], a["y"], a["total"], a["q"], a["s"], None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(cols=0), -1, "cols positive"), (dict(cols=20000), -2, "16384"), (dict(type=7), -1, "element type"),
    (dict(ttype=2), -1, "residual must be"), (dict(wtype=2), -1, "weight must be"),
    (dict(dx=None, dr=None, dw=None), -1, "no gradient"), (dict(ldt=8), -1, "ldt"), (dict(dy=None), -1, "dy is NULL"),
    (dict(t=ODD), -1, "total must be"), (dict(dt=ODD), -1, "dtotal"), (dict(dx=ODD), -1, "dx"),
    (dict(dr=ODD), -1, "dresidual"), (dict(dw=ODD), -1, "dweight"), (dict(ws=None), -1, "ws is NULL"),
    (dict(bytes=ctypes.c_size_t(16)), -3, "too small"),
])
def test_norm_gradient_refusals(lib, change, code, text):
    a = {**dict(dy=P, type=1, rows=4, cols=64, t=P, ttype=0, ldt=64, dt=P, w=P, wtype=1, dx=P, dr=P, dw=P, ws=P, bytes=BIG),
         **change}
    _refused(lib, lib.moe_rms_norm_backward(a["dy"], a["type"], a["rows"], a["cols"], a["t"], a["ttype"], a["ldt"], a["dt"],
                                            a["w"], a["wtype"], 1e-6, a["dx"], a["dr"], a["dw"], a["ws"], a["bytes"], None),
             code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(w=None), -1, "go together"), (dict(rw=None), -1, "go together"), (dict(idx=None), -1, "topk_idx is NULL"),
    (dict(counts=None), -1, "counts"), (dict(off=ODD), -1, "offsets"), (dict(inv=None), -1, "inv_pos"),
    (dict(tok=ODD), -1, "row_token"), (dict(rw=ODD), -1, "row_weight"), (dict(ws=None), -1, "ws is NULL"),
    (dict(bytes=ctypes.c_size_t(8)), -3, "too small"),
])
def test_sort_refusals(lib, change, code, text):
    a = {**dict(idx=P, w=P, counts=P, off=P, inv=P, tok=P, rw=P, ws=P, bytes=BIG), **change}
    _refused(lib, lib.moe_sort_tokens(ctypes.byref(_cfg(T=5000)), a["idx"], a["w"], a["counts"], a["off"], a["inv"], a["tok"],
                                      a["rw"], a["ws"], a["bytes"], None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(size=3), -1, "1, 2 or 4"), (dict(size=8), -1, "1, 2 or 4"), (dict(cols=0), -1, "positive"),
    (dict(cols=1 << 28), -2, "2^28"), (dict(ldx=63), -1, "ldx"), (dict(xs=P), -1, "go together"), (dict(x=None), -1, "x is"),
    (dict(inv=None), -1, "inv_pos"), (dict(off=None), -1, "offsets"), (dict(xd=ODD), -1, "xd"),
    (dict(xs=P, xds=ODD), -1, "xd_scales"),
])
def test_permute_refusals(lib, change, code, text):
    a = {**dict(x=P, size=2, cols=64, ldx=64, xs=None, inv=P, off=P, xd=P, xds=None), **change}
    _refused(lib, lib.moe_permute(ctypes.byref(_cfg()), a["x"], a["size"], a["cols"], a["ldx"], a["xs"], a["inv"], a["off"],
                                  a["xd"], a["xds"], None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(type=3), -1, "element type"), (dict(cols=-4), -1, "positive"), (dict(cols=1 << 30), -2, "2^28"),
    (dict(yd=None), -1, "yd"), (dict(inv=ODD), -1, "inv_pos"), (dict(y=None), -1, "is NULL"), (dict(w=ODD), -1, "weights"),
])
def test_unpermute_refusals(lib, change, code, text):
    a = {**dict(yd=P, type=1, cols=64, inv=P, w=P, y=P), **change}
    c = ctypes.byref(_cfg())
    _refused(lib, lib.moe_unpermute(c, a["yd"], a["type"], a["cols"], a["inv"], a["w"], None, a["y"], None), code, text)
    _refused(lib, lib.moe_unpermute_backward(c, a["y"], a["yd"], a["type"], a["cols"], a["inv"], P, a["w"], P, P, None),
             code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(type=2), -1, "fp32 or bf16"), (dict(logits=None), -1, "logits"), (dict(idx=ODD), -1, "topk_idx"),
    (dict(dw=None), -1, "dtopk_w"), (dict(out=ODD), -1, "dlogits"),
])
def test_route_gradient_refusals(lib, change, code, text):
    a = {**dict(logits=P, type=0, idx=P, dw=P, out=P), **change}
    _refused(lib, lib.moe_route_backward(ctypes.byref(_cfg()), a["logits"], a["type"], a["idx"], a["dw"], a["out"], None),
             code, text)


def test_nothing_to_do_returns_at_once(lib):
    c = ctypes.byref(_cfg(T=0))
    assert lib.moe_rms_norm(None, 1, 0, 64, 64, None, 1, 0, None, 1, 1e-6, P, None, None, None, None) == 0
    assert lib.moe_rms_norm_backward(None, 1, 0, 64, None, 1, 64, None, None, 1, 1e-6, P, None, None, None, 0, None) == 0
    assert lib.moe_permute(c, None, 2, 64, 64, None, None, None, None, None, None) == 0
    assert lib.moe_unpermute(c, None, 1, 64, None, None, None, None, None) == 0
    assert lib.moe_unpermute_backward(c, None, None, 1, 64, None, None, None, None, None, None) == 0
    assert lib.moe_route_backward(c, None, 0, None, None, None, None) == 0


def test_config_is_checked(lib):
    c = ctypes.byref(_cfg(k=9))
    assert lib.moe_permute(c, P, 2, 64, 64, None, P, P, P, None, None) == moe.MOE_ERR_INVALID
    assert lib.moe_route_backward(c, P, 0, P, P, P, None) == moe.MOE_ERR_INVALID
    assert lib.moe_sort_tokens(c, P, P, P, P, P, P, P, P, BIG, None) == moe.MOE_ERR_INVALID


def test_workspaces(lib):
    n = ctypes.c_size_t()
    for T, E, k in ((1, 8, 2), (70000, 256, 8), (1 << 20, 1024, 8)):  # a count of each expert for each block of assignments
        assert lib.moe_sort_tokens_workspace_size(ctypes.byref(_cfg(T=T, E=E, k=k)), ctypes.byref(n)) == 0
        blocks = -(-T * k // max(2048, -(-T * k // 128 // 2048) * 2048))
        assert (n.value == 0) if blocks == 1 else 4 * blocks * E <= n.value <= 4 * 129 * E
    for rows, cols in ((0, 5), (1, 16384), (100000, 7168), (100000, 3)):
        assert lib.moe_rms_norm_backward_workspace_size(rows, cols, ctypes.byref(n)) == 0
        assert n.value >= 4 * cols and n.value <= 4 * 152 * 32 * cols + 256
    assert lib.moe_rms_norm_backward_workspace_size(4, 4, None) == moe.MOE_ERR_INVALID
    assert lib.moe_rms_norm_backward_workspace_size(4, 0, ctypes.byref(n)) == moe.MOE_ERR_INVALID


def test_binding_checks_tensors():
    """Tensors of another device, type, shape or layout are refused by name before the library is called."""
    x, c = torch.zeros(64, 32), _cfg()
    idx = torch.zeros(64, 2, dtype=torch.int32)
    for call, name in ((lambda: moe.rms_norm(x), "x"), (lambda: moe.rms_norm_fp8(x), "x"),
                       (lambda: moe.rms_norm_backward(x, x), "dy"), (lambda: moe.sort_tokens(c, idx), "topk_idx"),
                       (lambda: moe.permute(c, x, idx, idx), "inv_pos"), (lambda: moe.unpermute(c, x, idx), "inv_pos"),
                       (lambda: moe.unpermute_backward(c, x, x, idx, idx), "inv_pos"),
                       (lambda: moe.route_weights(c, x), "logits"), (lambda: moe.route_backward(c, x, idx, x), "logits")):
        with pytest.raises(ValueError, match=f"^{name} must be a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="needs offsets"):
        moe.unpermute(c, x.requires_grad_(), idx)


# ------------------------------------------------------------------------------------------
# the definitions themselves
# ------------------------------------------------------------------------------------------
def _difference(f, v, step=1e-6):
    """Central differences of the number f(v) by every element of v (their error: step^2 times the third derivative, and
    rounding of about 1e-16 |f| / step)."""
    out = torch.zeros_like(v)
    for i in range(v.numel()):
        d = torch.zeros_like(v).view(-1)
        d[i] = step
        d = d.view(v.shape)
        out.view(-1)[i] = (f(v + d) - f(v - d)) / (2 * step)
    return out


def test_plain_norm_gradient_is_the_norms():
    g = torch.Generator().manual_seed(1)
    x, dy, dt = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(7, generator=g, dtype=torch.float64)
    f = lambda x, w: float((plain.norm(x, w, None, 1e-3)[0] * dy).sum() + (x * dt).sum())  # noqa: E731
    d, dw, _, _ = plain.norm_backward(dy, x, w, 1e-3, dt)
    assert (d - _difference(lambda v: f(v, w), x)).abs().max() < 1e-8
    assert (dw - _difference(lambda v: f(x, v), w)).abs().max() < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_plain_route_gradient_is_the_weights(score, renorm):
    g = torch.Generator().manual_seed(2)
    z = torch.randn(6, 5, generator=g, dtype=torch.float64)
    idx = torch.topk(z, 3).indices.int()
    idx[1, 2], idx[2], idx[3, 0] = -1, -1, 9
    idx[4, 1] = idx[4, 0]  # the same expert twice
    dw = torch.randn(6, 3, generator=g, dtype=torch.float64)
    f = lambda v: float((plain.route_weights(v, idx, score, renorm, 2.5).nan_to_num() * dw).sum())  # noqa: E731
    got, _ = plain.route_backward(z, idx, dw, score, renorm, 2.5)
    assert (got - _difference(f, z)).abs().max() < 1e-8


def test_plain_unpermute_gradient_is_the_sums():
    g = torch.Generator().manual_seed(3)
    idx = torch.tensor([[0, 1], [1, -1], [1, 1], [2, 0]], dtype=torch.int32)
    s = plain.sort(idx, 3, capacity=3)
    inv = torch.tensor(s["inv_pos"]).view(4, 2)
    assert s["counts"] == [2, 3, 1] and s["offsets"] == [0, 2, 5, 6]
    assert inv.tolist() == [[0, 2], [3, -1], [4, -1], [5, 1]] and s["row_token"] == [0, 3, 0, 1, 2, 3, -1, -1]
    yd, dy, w = (torch.randn(*n, generator=g, dtype=torch.float64) for n in ((8, 5), (4, 5), (4, 2)))
    f = lambda yd, w: float((plain.unpermute(yd, inv, w, None)[0] * dy).sum())  # noqa: E731
    dyd, dw, _ = plain.unpermute_backward(dy, yd, inv, w)
    assert (dyd - _difference(lambda v: f(v, w), yd)).abs().max() < 1e-8
    assert (dw - _difference(lambda v: f(yd, v), w)).abs().max() < 1e-8


def test_plain_sort_under_a_placement():
    idx = torch.tensor([[0], [0], [1], [0]], dtype=torch.int32)
    place = {"slot_expert": [0, 1, 0], "slot_replica": [1, 0, 0], "replicas": [2, 1], "replica_slot": None}
    s = plain.sort(idx, 2, placement=place)  # expert 0's rows go round slots 2 and 0
    assert s["counts"] == [1, 1, 2] and s["inv_pos"] == [2, 0, 1, 3]


def test_route_gradient_over_its_logits_is_refused(lib):
    c = ctypes.byref(_cfg())  # 64 x 8 fp32: 2048 bytes
    for off in (0, 16, 2032, -2032):
        out = ctypes.c_void_p(0x10000 + off)
        _refused(lib, lib.moe_route_backward(c, ctypes.c_void_p(0x10000), 0, P, P, out, None), -1, "overlaps")
