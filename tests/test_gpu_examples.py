"""The examples run, and do what they say."""
import importlib.util
import os

import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(EXAMPLES, name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rebalance_router(fmt):
    """The gradient evens the load: the loss falls towards its value for an even one (alpha = 1)."""
    pkg_build.build()
    rde.load()
    history, y = load("rebalance_router_fp4").main(steps=30, fmt=fmt)
    first, last = history[0], history[-1]
    assert last[0] < first[0] and last[0] - 1 < 0.5 * (first[0] - 1)
    assert last[1] < first[1]
    assert torch.isfinite(y.float()).all()
