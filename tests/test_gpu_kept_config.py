"""A configuration that changes between a forward and its backward pass: the gradient is that of the forward's."""
import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def _step(change):
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, E, k, cols = 24, 8, 2, 40
    cfg = rde.make_config(T=T, h=256, E=E, k=k, I=256, score="sigmoid", renorm=True, routed_scale=2.5)
    logits = torch.randn(T, E, generator=gen, device="cuda", requires_grad=True)
    x = torch.randn(T, cols, generator=gen, device="cuda", requires_grad=True)
    idx, w = rde.route_weights(cfg, logits)
    s = rde.sort_tokens(cfg, idx, w.detach())
    y = rde.unpermute(cfg, rde.permute(cfg, x, s["inv_pos"], s["offsets"]), s["inv_pos"], w, offsets=s["offsets"])
    if change:
        cfg.T, cfg.routed_scale, cfg.renormalize = 7, 1.0, 0
    (y * torch.randn(T, cols, generator=gen, device="cuda")).sum().backward()
    return logits.grad, x.grad


def test_configuration_changed_before_the_backward_pass():
    for a, b in zip(_step(False), _step(True)):
        assert torch.equal(a, b)
