"""Refusals of the 4-bit and balance-loss entry points that test_fp4_balance_host.py does not cover. No GPU: each call
returns before any CUDA call."""
import ctypes

import pytest
import torch

from routing_dispatch_expert_gb300 import moe
from test_fp4_balance_host import P, _cfg, _says, lib  # noqa: F401


@pytest.mark.parametrize("shared", [0, 256])
def test_mxfp4_layers_have_no_bf16_dispatch(lib, shared):  # noqa: F811
    """Rows in bf16 serve no MXFP4 entry point, and are four times what a caller with 4-bit rows has room for."""
    c = ctypes.byref(_cfg(dtype="mxfp4", I_shared=shared))
    big = ctypes.c_size_t(1 << 40)
    assert lib.moe_dispatch(c, P, P, P, P, P, P, P, P, P, None, P, big, None) == moe.MOE_ERR_UNSUPPORTED
    assert _says(lib, "_fp4 entry points")
    assert lib.moe_dispatch_noalloc(c, P, P, P, P, P, P, P, P, P, None, None) == moe.MOE_ERR_UNSUPPORTED
    assert _says(lib, "_fp4 entry points")


def test_balance_loss_refuses_what_is_no_cuda_tensor():
    """With and without a gradient, and things that are no tensors at all."""
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for logits in (torch.zeros(4, 8, requires_grad=True), torch.zeros(4, 8), [[0.0] * 8] * 4, None):
        with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
            moe.balance_loss(_cfg(T=4), logits, idx, 0.1)


def test_status_calls_check_their_arguments(lib):  # noqa: F811
    assert lib.moe_matmul_fp4_status(None, None) == moe.MOE_ERR_INVALID
    assert _says(lib, "status")
    c = ctypes.byref(_cfg())
    assert lib.moe_selftest_wait_timeout(c, None, 0, 0, None) == moe.MOE_ERR_INVALID  # the limit, not ws
    assert _says(lib, "limit_cycles")
    assert lib.moe_selftest_wait_timeout(c, P, 16, 1000, None) == moe.MOE_ERR_WORKSPACE
