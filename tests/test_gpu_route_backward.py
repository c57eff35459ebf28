"""The route weights' gradient on the GPU. Errors relative to the sums of magnitudes that plain_rows gives: an exponential is
2 ulp (4 u) and carries its argument's rounding, u times an argument of at most about 20 here; a score adds a division and a
sum over the experts (at most 32 + 5 + 32 additions, all positive) and the result two sums over k <= 32 slots and five
products: below 160 u."""
import pytest
import torch

import plain_rows as plain
import routing_dispatch_expert_gb300 as rde
from plain_rows import HALF, TINY, U32
from routing_dispatch_expert_gb300 import build as pkg_build
from test_gpu_rms_norm import close

pytestmark = pytest.mark.gpu
MODES = [(s, r) for s in ("softmax", "sigmoid") for r in (False, True)]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def config(T, E, k, score, renorm, **kw):
    return rde.make_config(T=T, h=256, E=E, k=k, I=256, score=score, renorm=renorm, routed_scale=2.5, **kw)


def inputs(T, E, k, dtype=torch.float32, seed=0, twice=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn(T, E, generator=gen, device="cuda") * 2).to(dtype)
    idx = torch.topk(z.float(), k).indices.int()
    if twice:
        idx = torch.randint(-1, E + 1, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    return z, idx.contiguous(), torch.randn(T, k, generator=gen, device="cuda")


def check(cfg, z, idx, dw, score, renorm):
    got = rde.route_backward(cfg, z, idx, dw)
    want, size = plain.route_backward(z.cpu(), idx.cpu(), dw.cpu(), score, renorm, 2.5)
    assert got.dtype == z.dtype
    close(got.cpu(), want, 160 * U32 * size + HALF[z.dtype] * want.abs() * (1 + 2.0 ** -8) + TINY[z.dtype], "dlogits")
    return got


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 2, 2), (33, 8, 2), (33, 8, 8), (9, 7, 5), (40, 13, 13), (20, 60, 6), (17, 64, 32),
                                   (12, 127, 4), (9, 128, 8), (30, 256, 8), (5, 300, 31), (6, 512, 8), (4, 1023, 8), (3, 1024, 32)])
def test_gradient(score, renorm, T, E, k):
    for dtype in (torch.float32, torch.bfloat16):
        for twice in (False, True):
            check(config(T, E, k, score, renorm), *inputs(T, E, k, dtype, E + k, twice), score, renorm)


@pytest.mark.parametrize("score,renorm", MODES)
def test_many_tokens(score, renorm):
    """More tokens than one round of the grid: the same rows again and again."""
    T, E, k, n = 16, 16, 4, 9001
    z, idx, dw = inputs(T, E, k)
    one = check(config(T, E, k, score, renorm), z, idx, dw, score, renorm)
    many = rde.route_backward(config(T * n, E, k, score, renorm), z.repeat(n, 1), idx.repeat(n, 1), dw.repeat(n, 1))
    assert torch.equal(many, one.repeat(n, 1))


@pytest.mark.parametrize("score,renorm", MODES)
def test_rows_without_choices_and_masked_experts(score, renorm):
    T, E, k = 8, 12, 3
    z, idx, dw = inputs(T, E, k)
    z[1, 4:] = -float("inf")       # masked experts that are not chosen
    idx[1] = torch.tensor([0, 1, 2])
    idx[2] = -1                    # a padded token, with anything in its row
    z[2], dw[2] = float("nan"), float("nan")
    z[3] = -float("inf")           # nothing but masked experts
    idx[4, 1:] = 99
    dw[4, 1:] = float("nan")
    z[5] -= 300                    # sigmoids that all underflow
    z[6] += 300
    got = rde.route_backward(config(T, E, k, score, renorm), z, idx, dw)
    assert torch.isfinite(got).all() and (got[2] == 0).all() and (got[3] == 0).all()
    assert (got[1, 4:] == 0).all()
    if renorm:  # a shift of all logits leaves a softmax, and sigmoids that are e^l, as they are
        ref = torch.softmax(z[5, idx[5].long()].double(), 0)
        d = 2.5 * ref * (dw[5].double() - (ref * dw[5].double()).sum())
        assert torch.allclose(got[5, idx[5].long()].double(), d, rtol=0, atol=1e-3 * float(dw[5].abs().max()))


@pytest.mark.parametrize("score,renorm", MODES)
def test_autograd_of_the_routers_own_weights(score, renorm):
    T, E, k = 60, 32, 4
    cfg = config(T, E, k, score, renorm)
    z, _, dw = inputs(T, E, k)
    bias = torch.randn(E, device="cuda") * 0.1 if score == "sigmoid" else None
    a = z.clone().requires_grad_()
    idx, w = rde.route_weights(cfg, a, bias)
    (w * dw).sum().backward()
    assert not idx.requires_grad and torch.equal(a.grad, check(cfg, z, idx, dw, score, renorm))
    want = plain.route_weights(z, idx, score, renorm, 2.5)
    assert torch.allclose(w.detach().double(), want, rtol=4e-6, atol=0)
    with torch.no_grad():
        assert not rde.route_weights(cfg, a, bias)[1].requires_grad


@pytest.mark.parametrize("score,renorm", MODES)
def test_gradient_by_differences(score, renorm):
    """Differences of the library's own weights (fp32) for fixed choices: a step of 2^-5 leaves h^2 / 6 of a third derivative
    of about the weights' size and 2^-22 / h of them."""
    T, E, k = 4, 8, 3
    cfg = config(T, E, k, score, renorm)
    z, _, dw = inputs(T, E, k, seed=3)
    z = (z * 0.5).contiguous()
    idx, w = rde.route_weights(cfg, z)
    z.scatter_add_(1, idx.long(), torch.full((T, k), 2.0, device="cuda"))  # far enough that the choice stays
    idx, w = rde.route_weights(cfg, z)
    d = rde.route_backward(cfg, z, idx, dw)
    h = 2.0 ** -5

    def f(v):
        i, w = rde.route_weights(cfg, v)
        order = (i.unsqueeze(1) == idx.unsqueeze(2)).float().argmax(2)  # slot j's expert, wherever it now stands
        return (w.gather(1, order).double() * dw.double()).sum(1)

    for e in range(E):
        step = torch.zeros_like(z)
        step[:, e] = h
        got = (f(z + step) - f(z - step)) / (2 * h)
        assert (got - d[:, e].double()).abs().max() < 1e-3 * 2.5 * float(dw.abs().max()) * k
