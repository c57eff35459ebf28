"""The sort at the sizes where its blocks change: the same order as numpy's stable sort, and one launch or two."""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build
from test_gpu_permute import choices, config

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


@pytest.mark.parametrize("T,E,k", [(128, 256, 8), (1023, 9, 1), (1024, 9, 1), (1025, 9, 1), (1024, 8, 2), (683, 8, 3), (2049, 1024, 1),
                                   (2048, 1024, 8), (2049, 1024, 8), (8192, 256, 8), (8193, 256, 8), (16384, 64, 8),
                                   (16385, 64, 8), (65536, 3, 2), (65537, 3, 2)])
@pytest.mark.parametrize("pad", [0.0, 0.4])
def test_sort(T, E, k, pad):
    idx, w = choices(T, E, k, seed=T, pad=pad), torch.rand(T, k, device="cuda")
    cfg = config(T, E, k)
    rde.sort_tokens(cfg, idx, w)
    before = rde.launch_count()
    got = rde.sort_tokens(cfg, idx, w)
    assert rde.launch_count() - before == (1 if T * k <= 2048 else 2)
    flat = idx.flatten().cpu().numpy()
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:(flat >= 0).sum()]
    inv = np.full(T * k, -1, np.int32)
    inv[order] = np.arange(order.size, dtype=np.int32)
    np.testing.assert_array_equal(got["inv_pos"].flatten().cpu().numpy(), inv)
    np.testing.assert_array_equal(got["row_token"].cpu().numpy()[:order.size], order // k)
    np.testing.assert_array_equal(got["row_weight"].cpu().numpy()[:order.size], w.flatten().cpu().numpy()[order])
    assert (got["row_token"][order.size:] == -1).all() and (got["row_weight"][order.size:] == 0).all()
    np.testing.assert_array_equal(got["counts"].cpu().numpy(), np.bincount(flat[flat >= 0], minlength=E))
    np.testing.assert_array_equal(got["offsets"].cpu().numpy(), np.concatenate(([0], np.cumsum(got["counts"].cpu().numpy()))))
