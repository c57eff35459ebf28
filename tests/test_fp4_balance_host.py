"""The 4-bit and balance-loss entry points without a GPU: their refusals (each returns before any CUDA
call), workspace sizes, the binding's checks, and the 64-bit definitions that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import plain_fp4 as plain
from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe

P = ctypes.c_void_p(0x1000)  # aligned, never read: the calls fail before
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return moe.load()


def _cfg(**kw):
    return moe.make_config(**{**dict(T=64, h=256, E=8, k=2, I=256, dtype="nvfp4"), **kw})


def _says(lib, text):
    return text in lib.moe_last_error().decode()


@pytest.mark.parametrize("change,code,text", [
    (dict(rows=-1), -1, "negative"), (dict(cols=48), -2, "multiple of 32"), (dict(fmt=2), -1, "format"),
    (dict(type=3), -1, "type"), (dict(ldx=32), -1, "ldx"), (dict(ldx=68), -1, "16-byte"),
    (dict(type=0, ldx=66), -1, "16-byte"), (dict(x=None), -1, "NULL"), (dict(q=ODD), -1, "aligned"),
    (dict(s=None), -1, "NULL"), (dict(rows=1 << 40, ldx=64), -2, "2^32"),
])
def test_quantize_refusals(lib, change, code, text):
    a = {**dict(x=P, type=1, rows=4, cols=64, ldx=64, fmt=0, g=None, q=P, s=P), **change}
    assert lib.moe_quantize_fp4(a["x"], a["type"], a["rows"], a["cols"], a["ldx"], a["fmt"], a["g"], a["q"], a["s"],
                                None) == code
    assert _says(lib, text)


def test_nothing_to_do_returns_at_once(lib):
    assert lib.moe_quantize_fp4(None, 1, 0, 64, 64, 0, None, None, None, None) == 0
    assert lib.moe_quantize_fp4(None, 1, 4, 0, 0, 1, None, None, None, None) == 0
    assert lib.moe_dequantize_fp4(None, None, 0, 64, 0, None, 0, None, None) == 0
    assert lib.moe_matmul_fp4(None, None, None, None, None, None, 0, 8, 32, 0, 1, None, 8, None, None) == 0
    assert lib.moe_balance_loss_backward(ctypes.byref(_cfg(T=0)), None, 0, None, None, None, 1, None, 0.1, None, None,
                                         None) == 0


@pytest.mark.parametrize("change,code,text", [
    (dict(fmt=-1), -1, "format"), (dict(type=9), -1, "type"), (dict(cols=16), -2, "multiple of 32"),
    (dict(q=None), -1, "NULL"), (dict(y=ODD), -1, "aligned"),
])
def test_dequantize_refusals(lib, change, code, text):
    a = {**dict(q=P, s=P, rows=4, cols=64, fmt=1, type=0, y=P), **change}
    assert lib.moe_dequantize_fp4(a["q"], a["s"], a["rows"], a["cols"], a["fmt"], None, a["type"], a["y"], None) == code
    assert _says(lib, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(M=-1), -1, "positive"), (dict(N=0), -1, "positive"), (dict(K=0), -1, "positive"), (dict(K=40), -2, "32"),
    (dict(fmt=5), -1, "format"), (dict(type=2), -1, "bf16 or fp32"), (dict(ldy=7), -1, "ldy"),
    (dict(M=1 << 31), -2, "too large"), (dict(M=1 << 30, N=1 << 20, ldy=1 << 20), -2, "too large"),
    (dict(aq=None), -1, "NULL"), (dict(bs=ODD), -1, "aligned"), (dict(y=None), -1, "NULL"),
])
def test_matmul_refusals(lib, change, code, text):
    a = {**dict(aq=P, as_=P, bq=P, bs=P, M=4, N=8, K=64, fmt=0, type=1, y=P, ldy=8), **change}
    assert lib.moe_matmul_fp4(a["aq"], a["as_"], None, a["bq"], a["bs"], None, a["M"], a["N"], a["K"], a["fmt"],
                              a["type"], a["y"], a["ldy"], None, None) == code
    assert _says(lib, text)


def test_layer_refusals(lib):
    big = ctypes.c_size_t(1 << 40)
    w = moe.MoeWeightsStruct()
    for f in ("w_router", "w_gu", "w_d", "s_gu", "s_d", "g_gu", "g_d"):
        setattr(w, f, 0x1000)
    for dtype in ("bf16", "fp8"):  # rows of 4 bits need weights of 4 bits
        c = _cfg(dtype=dtype)
        assert lib.moe_forward_fp4(ctypes.byref(c), P, ctypes.byref(w), None, P, P, big, None) == moe.MOE_ERR_UNSUPPORTED
        assert _says(lib, "4-bit rows need")
    c = _cfg(dtype="mxfp4")  # and weights of MXFP4 have no other path
    assert lib.moe_forward(ctypes.byref(c), P, ctypes.byref(w), P, P, big, None) == moe.MOE_ERR_UNSUPPORTED
    assert _says(lib, "_fp4 entry points")
    assert lib.moe_expert_ffn(ctypes.byref(c), ctypes.byref(w), P, None, P, P, P, P, big, None) == moe.MOE_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.moe_workspace_size(ctypes.byref(_cfg(dtype="mxfp4", I=128)), ctypes.byref(n)) == moe.MOE_ERR_UNSUPPORTED
    c = _cfg()
    assert lib.moe_forward_fp4(ctypes.byref(c), P, ctypes.byref(w), None, P, P, 16, None) == moe.MOE_ERR_WORKSPACE
    assert lib.moe_forward_fp4(ctypes.byref(c), None, ctypes.byref(w), None, P, P, big, None) == moe.MOE_ERR_INVALID
    assert lib.moe_expert_ffn_fp4(ctypes.byref(c), ctypes.byref(w), None, P, None, P, P, P, P, big,
                                  None) == moe.MOE_ERR_INVALID
    assert _says(lib, "xs is NULL")
    assert lib.moe_dispatch_fp4(ctypes.byref(c), None, P, P, P, P, P, P, P, P, P, ODD, P, big,
                                None) == moe.MOE_ERR_INVALID
    w.g_d = None  # NVFP4 weights have matrix scales
    assert lib.moe_forward_fp4(ctypes.byref(c), P, ctypes.byref(w), None, P, P, big, None) == moe.MOE_ERR_INVALID
    assert _says(lib, "g_gu / g_d")


@pytest.mark.parametrize("change,code,text", [
    (dict(type=2), -1, "fp32 or bf16"), (dict(S=0), -1, "n_seq"), (dict(S=2, off=None), -1, "seq_offsets"),
    (dict(S=(1 << 24) + 1), -2, "n_seq"), (dict(logits=None), -1, "NULL"), (dict(idx=ODD), -1, "aligned"),
    (dict(loss=None), -1, "NULL"), (dict(bytes=16), -3, "workspace"),
])
def test_balance_loss_refusals(lib, change, code, text):
    a = {**dict(logits=P, type=0, idx=P, off=P, S=3, loss=P, bytes=1 << 30), **change}
    c = _cfg()
    assert lib.moe_balance_loss(ctypes.byref(c), a["logits"], a["type"], a["idx"], a["off"], a["S"], None, 0.1, a["loss"],
                                P, P, P, P, a["bytes"], None) == code
    assert _says(lib, text)
    if "idx" not in change and "loss" not in change and "bytes" not in change:
        assert lib.moe_balance_loss_backward(ctypes.byref(c), a["logits"], a["type"], P, P, a["off"], a["S"], None, 0.1,
                                             P, P, None) == code


def test_balance_loss_workspace_holds_every_block_and_sequence(lib):
    """One entry of 2 E + 1 words for each block of tokens and each sequence."""
    for T, E, S in ((1, 2, 1), (70000, 256, 1), (512, 1024, 300)):
        n = ctypes.c_size_t()
        assert lib.moe_balance_loss_workspace_size(ctypes.byref(_cfg(T=T, E=E)), S, ctypes.byref(n)) == 0
        assert n.value >= 4 * (2 * E + 1) * (S + 1)
    assert lib.moe_balance_loss_workspace_size(ctypes.byref(_cfg()), 1, None) == moe.MOE_ERR_INVALID


def test_binding_checks_tensors():
    """Tensors of another device, type, shape or layout are refused by name before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        moe.quantize_fp4(x)
    with pytest.raises(ValueError, match="unknown 4-bit format"):
        moe.quantize_fp4(x, "fp4")
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        moe.balance_loss(_cfg(T=4), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 0.1)


# ------------------------------------------------------------------------------------------
# the definitions themselves
# ------------------------------------------------------------------------------------------
def test_plain_nvfp4_is_the_weight_quantisers_format():
    """The definition of the tests equals the fp64 oracle's NVFP4, which the weight quantiser is held to."""
    rng = np.random.default_rng(3)
    w = torch.from_numpy(rng.normal(0, 0.02, (24, 256))).to(torch.bfloat16)
    w[3] = 0
    w[5, 16:32] = 1e-30
    bits = w.view(torch.int16).numpy().view(np.uint16)
    q, s, g = oracle.quant_weight_nvfp4(bits)
    pq, ps = plain.quantize(w, "nvfp4", float(g))
    np.testing.assert_array_equal(pq.numpy(), q)
    np.testing.assert_array_equal(ps.numpy(), s)
    np.testing.assert_array_equal(plain.values(pq, ps, "nvfp4", float(g)).numpy(), oracle.dequant_nvfp4(q, s, g))


def test_plain_mxfp4_by_hand():
    x = torch.zeros(1, 64)
    x[0, :8] = torch.tensor([8.0, -4.0, 0.25, -0.25, 5.0, 7.0, 0.75, 3.0])  # scale 2^(3 - 2) = 2
    q, s = plain.quantize(x, "mxfp4")
    assert s.tolist() == [[128, 0]]  # and 2^-127 for a block of zeros
    assert plain.values(q, s, "mxfp4")[0, :8].tolist() == [8.0, -4.0, 0.0, 0.0, 4.0, 8.0, 1.0, 3.0]
    x[0, 40] = float("inf")
    q, s = plain.quantize(x, "mxfp4")
    assert s.tolist() == [[128, 255]] and torch.isnan(plain.values(q, s, "mxfp4")[0, 32:]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_plain_gradient_is_the_losses(score):
    """The formula of the gradient against central differences of the loss (step 1e-5: the error of a difference
    is about step^2 times the third derivative, and 1e-16 / step of rounding: below 1e-9 here)."""
    rng = torch.Generator().manual_seed(7)
    T, E, k = 13, 5, 2
    logits = torch.randn(T, E, generator=rng, dtype=torch.float64)
    idx = torch.topk(logits, k).indices.int()
    off, mask = [0, 4, 4, 11], torch.rand(T, generator=rng) > 0.2
    dloss = torch.tensor([1.0, 2.0, -0.5], dtype=torch.float64)
    counts = plain.balance_loss(logits, idx, score, 0.3, off, mask)["counts"]
    got = plain.balance_loss_backward(logits, counts, k, score, 0.3, dloss, off, mask)
    f = lambda z: float((plain.balance_loss(z, idx, score, 0.3, off, mask)["loss"] * dloss).sum())  # noqa: E731
    for t in range(T):
        for e in range(E):
            d = torch.zeros(T, E, dtype=torch.float64)
            d[t, e] = 1e-5
            assert abs((f(logits + d) - f(logits - d)) / 2e-5 - float(got[t, e])) < 1e-8


def test_even_load_has_loss_alpha():
    E, k, T = 8, 2, 32
    idx = (torch.arange(T * k).view(T, k) % E).int()
    out = plain.balance_loss(torch.zeros(T, E), idx, "softmax", 0.25)
    assert abs(float(out["loss"]) - 0.25) < 1e-12 and out["counts"].tolist() == [[T * k // E] * E]
