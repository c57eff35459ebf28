"""The sort's workspace: a size that never falls as the batch grows, and that the largest batch's serves smaller ones."""
import ctypes

import numpy as np
import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    pkg_build.build()
    return moe.load()


def size(T, E, k):
    n = ctypes.c_size_t()
    assert moe.load().moe_sort_tokens_workspace_size(ctypes.byref(rde.make_config(T, 256, E, k, 256)), ctypes.byref(n)) == 0
    return n.value


def blocks(n, E):
    """Blocks of the sort: 1024 assignments a round of each where that makes few blocks, else 2048, 128 blocks at most."""
    two = n <= 1024 or (n > 2048 and n <= 131072 and n * E <= 1 << 24)
    items = 1024 if two else 2048
    return -(-n // max(items, -(-(-(-n // 128)) // items) * items))


@pytest.mark.parametrize("E", [8, 33, 64, 256, 1000, 1024])
@pytest.mark.parametrize("k", [1, 8])
def test_size_never_falls(E, k):
    switches = [0, 1024, 2048, 2 ** 24 // E, 131072, 128 * 2048, 2 * 128 * 2048, 5 * 128 * 1024]  # numbers of assignments
    T = sorted({max(0, n // k + d) for n in switches for d in (-2, -1, 0, 1, 2)} | set(range(0, 300000 // k, 4999 // k)))
    sizes = [size(t, E, k) for t in T]
    assert sizes == sorted(sizes)
    for t, s in zip(T, sizes):
        n = t * k
        assert (s == 0) == (n <= 2048) == (blocks(n, E) <= 1)
        if s:
            assert 4 * E * blocks(n, E) <= s <= 4 * E * min(128, -(-n // 1024)) + 255
    assert all(size(5000, e, k) <= size(5000, e + 1, k) for e in range(8, 300, 7))


def test_norm_gradient_size_never_falls(lib):
    n = ctypes.c_size_t()
    for cols in (1, 33, 255, 257, 1000, 4101, 7168, 16384):
        last = 0
        for rows in list(range(0, 3000, 7)) + [4864, 4865, 10 ** 5, 10 ** 6]:
            assert lib.moe_rms_norm_backward_workspace_size(rows, cols, ctypes.byref(n)) == 0
            assert n.value >= last
            last = n.value


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,largest,smaller", [(256, 8, 12000, (8193, 8192, 8191, 4096, 257, 256, 100, 1)),
                                                 (1024, 8, 2049, (2048, 2047, 300)), (64, 8, 16385, (16384, 3000)),
                                                 (8, 1, 262145, (262144, 131073, 131072, 2049))])
def test_the_largest_batchs_workspace_serves_smaller_ones(E, k, largest, smaller):
    ws = rde.sort_tokens_workspace(rde.make_config(largest, 256, E, k, 256))
    gen = torch.Generator(device="cuda").manual_seed(E)
    for T in (largest, *smaller):
        idx = torch.randint(0, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
        got = rde.sort_tokens(rde.make_config(T, 256, E, k, 256), idx, ws=ws)
        order = np.argsort(idx.flatten().cpu().numpy(), kind="stable")
        np.testing.assert_array_equal(got["row_token"].cpu().numpy(), order // k)
