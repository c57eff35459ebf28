"""The balance loss as a node of autograd: the gradient that reaches the logits is balance_loss_backward's."""
import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from test_gpu_balance_loss import ALPHA, built, config, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


def manual(cfg, logits, idx, off, mask, dloss):
    out = rde.balance_loss(cfg, logits.detach(), idx, ALPHA, off, mask)
    return out, rde.balance_loss_backward(cfg, logits.detach(), out["counts"], out["tokens"], ALPHA, dloss, off, mask)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,seqs", [(1, 8, 1), (70, 12, 3), (9000, 64, 5)])
def test_backward(score, dtype, T, E, seqs):
    cfg = config(T, E, 2, score)
    logits, idx, off, mask = inputs(T, E, 2, dtype, seqs=seqs, pad=0.1)
    for weight in (None, torch.rand(seqs, device="cuda")):
        dloss = torch.ones(seqs, device="cuda") if weight is None else weight
        want, dwant = manual(cfg, logits, idx, off, mask, dloss)
        z = logits.clone().requires_grad_()
        out = rde.balance_loss(cfg, z, idx, ALPHA, off, mask)
        assert all(torch.equal(out[m], want[m]) for m in want)
        assert out["loss"].requires_grad and not out["mean_prob"].requires_grad
        (out["loss"].sum() if weight is None else (out["loss"] * weight).sum()).backward()  # an expanded and a real dloss
        assert z.grad.dtype == dtype and torch.equal(z.grad, dwant)


def test_gradient_of_a_slice_of_other_losses():
    """A gradient that arrives as a slice, not 16-byte aligned."""
    T, E, seqs = 300, 8, 3
    cfg = config(T, E, 2, "softmax")
    logits, idx, off, mask = inputs(T, E, 2, torch.float32, seqs=seqs)
    weight = torch.rand(seqs + 1, device="cuda")
    _, dwant = manual(cfg, logits, idx, off, mask, weight[1:].clone())
    z = logits.clone().requires_grad_()
    out = rde.balance_loss(cfg, z, idx, ALPHA, off, mask)
    (torch.cat((torch.zeros(1, device="cuda"), out["loss"])) * weight).sum().backward()
    assert torch.equal(z.grad, dwant)


def test_through_a_router_weight_and_without_gradients():
    T, E, h = 500, 16, 32
    cfg = config(T, E, 2, "softmax")
    x = torch.randn(T, h, device="cuda")
    w = torch.randn(E, h, device="cuda", requires_grad=True)
    logits = x @ w.T
    idx = torch.topk(logits, 2).indices.int()
    out = rde.balance_loss(cfg, logits, idx, ALPHA)
    out["loss"].backward()
    _, d = manual(cfg, logits, idx, None, None, torch.ones(1, device="cuda"))
    assert torch.allclose(w.grad, d.T @ x, rtol=1e-5, atol=1e-9)
    with torch.no_grad():
        assert not rde.balance_loss(cfg, logits, idx, ALPHA)["loss"].requires_grad
    assert not rde.balance_loss(cfg, logits.detach(), idx, ALPHA)["loss"].requires_grad


def test_only_one_derivative_and_saved_logits_are_guarded():
    T, E = 64, 8
    cfg = config(T, E, 2, "sigmoid")
    logits, idx, _, _ = inputs(T, E, 2, torch.float32)
    z = logits.clone().requires_grad_()
    d, = torch.autograd.grad(rde.balance_loss(cfg, z, idx, ALPHA)["loss"].sum(), z, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()
    y = z * 1.0
    loss = rde.balance_loss(cfg, y, idx, ALPHA)["loss"]
    y.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_captured_step_and_another_stream():
    """Loss and gradient of a step captured into a graph, and of a step on a stream of its own: the same bits."""
    T, E, seqs = 4000, 64, 4
    cfg = config(T, E, 4, "sigmoid")
    logits, idx, off, mask = inputs(T, E, 4, torch.float32, seqs=seqs, pad=0.1)
    _, dwant = manual(cfg, logits, idx, off, mask, torch.ones(seqs, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = logits.clone().requires_grad_()
        rde.balance_loss(cfg, z, idx, ALPHA, off, mask)["loss"].sum().backward()
        assert torch.equal(z.grad, dwant)
        z = torch.zeros_like(logits, requires_grad=True)
        grad = torch.zeros_like(logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = rde.balance_loss(cfg, z, idx, ALPHA, off, mask)["loss"]
        grad.copy_(torch.autograd.grad(loss.sum(), z)[0])
    with torch.no_grad():
        z.copy_(logits)
    graph.replay()
    assert torch.equal(grad, dwant)
