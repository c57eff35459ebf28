"""Normalised sigmoid weights of logits far below zero, whose sigmoids all underflow in fp32: their ratios are those of the
definition in 64 bits, as the routing gradient takes them too.

Tolerance: a score is off by 4e-7 of itself (the exponential's 2 ulp and two operations), so is their sum, which takes k - 1 roundings
more; the quotient and the product two. Scores below 2^-149 are lost beside a sum of at least 1e-26: 2.5 * 2^-149 / 1e-26 is below
1e-12, absolutely."""
import pytest
import torch

import plain_rows as plain
import routing_dispatch_expert_gb300 as rde
from plain_rows import U32
from routing_dispatch_expert_gb300 import build as pkg_build
from test_gpu_rms_norm import close

pytestmark = pytest.mark.gpu
SHIFTS = [0, -20, -50, -57, -59, -60, -61, -75, -87, -88, -89, -95, -104, -150, -300, -600]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def check(w, z, idx, k):
    want = plain.route_weights(z, idx, "sigmoid", True, 2.5)
    assert torch.isfinite(w).all() and torch.isfinite(want).all()
    close(w, want, (2 * 4e-7 + (k + 2) * U32) * want + 1e-12, "weights")


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (60, 6), (64, 32), (256, 8), (1024, 8)])
@pytest.mark.parametrize("shift", SHIFTS)
def test_route_weights(E, k, shift):
    gen = torch.Generator(device="cuda").manual_seed(E)
    T = 40
    cfg = rde.make_config(T=T, h=256, E=E, k=k, I=256, score="sigmoid", renorm=True, routed_scale=2.5)
    for spread in (1.0, 4.0, 20.0):
        z = torch.randn(T, E, generator=gen, device="cuda") * spread + shift
        z[3] = shift  # all the same
        if E > k:
            z[4, k:] = -float("inf")  # masked experts
        z.requires_grad_()
        idx, w = rde.route_weights(cfg, z)
        check(w.detach(), z.detach(), idx, k)
        dw = torch.randn(T, k, generator=gen, device="cuda")
        w.backward(dw)
        assert torch.isfinite(z.grad).all() and torch.equal(z.grad, rde.route_backward(cfg, z.detach(), idx, dw))


@pytest.mark.parametrize("T", [8, 64, 3000])
@pytest.mark.parametrize("E,k,n_group", [(16, 4, 1), (128, 8, 4)])
def test_layer(T, E, k, n_group):
    """The whole layer, by its fused route and dispatch for few tokens and by the steps for more."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    h = I = 256
    x = torch.rand(T, h, generator=gen, device="cuda").to(torch.bfloat16) + 0.5
    w_r = -torch.rand(E, h, generator=gen, device="cuda") * 0.1 - 0.5  # logits of about -140
    rnd = lambda *n: (torch.randn(*n, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)  # noqa: E731
    cfg = rde.make_config(T=T, h=h, E=E, k=k, I=I, n_group=n_group, topk_group=max(1, n_group // 2), score="sigmoid", renorm=True,
                          routed_scale=2.5)
    layer = rde.MoeLayer(cfg, rde.Weights(w_router=w_r, w_gu=rnd(E, 2 * I, h), w_d=rnd(E, h, I)))
    y = layer(x)
    z = rde.ws_view(layer.ws, cfg, "logits", torch.float32, (T, E))
    idx = rde.ws_view(layer.ws, cfg, "topk_idx", torch.int32, (T, k))
    assert (z < -90).all() and torch.isfinite(y).all() and (y != 0).any()
    check(rde.ws_view(layer.ws, cfg, "topk_w", torch.float32, (T, k)), z, idx, k)
