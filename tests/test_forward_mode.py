"""Forward-mode derivatives: no call takes one, so each refuses a tensor that has a tangent, instead of giving an output
without one, which stands for a derivative of zero. The refusals come before any CUDA call."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from routing_dispatch_expert_gb300 import moe


def calls(make, device):
    """(name of the call, call) for each argument that may have a tangent; make(...): a tensor with one."""
    cfg = moe.make_config(T=4, h=256, E=8, k=2, I=256)
    x, w, tw = torch.randn(4, 16, device=device), torch.ones(16, device=device), torch.ones(4, 2, device=device)
    idx = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device=device)
    off = torch.arange(9, dtype=torch.int32, device=device)
    z, yd = torch.randn(4, 8, device=device), torch.randn(8, 16, device=device)
    yield "rms_norm x", lambda: moe.rms_norm(make(x), w)
    yield "rms_norm weight", lambda: moe.rms_norm(x, make(w))
    yield "rms_norm residual", lambda: moe.rms_norm(x, w, make(x))
    yield "rms_norm_fp8", lambda: moe.rms_norm_fp8(make(x), with_y=True)
    yield "rms_norm_backward dy", lambda: moe.rms_norm_backward(make(x), x, w)
    yield "rms_norm_backward total", lambda: moe.rms_norm_backward(x, make(x))
    yield "rms_norm_backward dtotal", lambda: moe.rms_norm_backward(x, x, w, dtotal=make(x))
    yield "sort_tokens", lambda: moe.sort_tokens(cfg, idx, make(tw))
    yield "permute", lambda: moe.permute(cfg, make(x), idx, off)
    yield "unpermute yd", lambda: moe.unpermute(cfg, make(yd), idx, tw)
    yield "unpermute weights", lambda: moe.unpermute(cfg, yd, idx, make(tw))
    yield "unpermute base", lambda: moe.unpermute(cfg, yd, idx, tw, make(x))
    yield "unpermute_backward dy", lambda: moe.unpermute_backward(cfg, make(x), yd, idx, off)
    yield "unpermute_backward yd", lambda: moe.unpermute_backward(cfg, x, make(yd), idx, off)
    yield "route_weights", lambda: moe.route_weights(cfg, make(z))
    yield "route_backward logits", lambda: moe.route_backward(cfg, make(z), idx, tw)
    yield "route_backward dtopk_w", lambda: moe.route_backward(cfg, z, idx, make(tw))
    yield "balance_loss", lambda: moe.balance_loss(cfg, make(z), idx, 0.1)


def check(device):
    from routing_dispatch_expert_gb300 import build as pkg_build

    pkg_build.build()
    moe.load()
    with forward_ad.dual_level():
        for grad in (False, True):
            make = lambda t: forward_ad.make_dual(t.clone().requires_grad_(grad), torch.ones_like(t))  # noqa: E731
            for name, call in calls(make, device):
                before = moe.launch_count()
                with torch.set_grad_enabled(False):  # forward mode stays on without a graph
                    with pytest.raises(NotImplementedError, match="forward-mode"):
                        call()
                assert moe.launch_count() == before, name
                if not grad:
                    with pytest.raises(NotImplementedError, match="forward-mode"):
                        call()


def test_tangents_are_refused():
    check("cpu")


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu():
    check("cuda")


@pytest.mark.gpu
def test_tangents_of_leaves_are_refused_by_autograd():
    """With a graph the call goes through its node, which has no forward-mode rule either."""
    with forward_ad.dual_level():
        x = forward_ad.make_dual(torch.randn(4, 16, device="cuda", requires_grad=True), torch.ones(4, 16, device="cuda"))
        with pytest.raises(NotImplementedError):
            moe.rms_norm(x)


@pytest.mark.gpu
def test_others_are_taken_in_an_open_level():
    x = torch.randn(4, 16, device="cuda")
    want = moe.rms_norm(x)
    with forward_ad.dual_level():
        assert torch.equal(moe.rms_norm(x), want)
        d = forward_ad.make_dual(x, torch.ones_like(x))
        assert torch.equal(moe.rms_norm(x), want)  # the primal itself has no tangent
        with torch.inference_mode():  # nothing is derived here
            assert torch.equal(moe.rms_norm(d), want)
        assert torch.equal(moe.rms_norm(forward_ad.unpack_dual(d).primal), want)
    assert torch.equal(moe.rms_norm(x), want)


def test_sorted_weights_that_require_a_gradient_are_refused():
    """The sort has no gradient in either mode: its row_weight would cut the router's."""
    cfg = moe.make_config(T=4, h=256, E=8, k=2, I=256)
    idx, w = torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, 2, requires_grad=True)
    with pytest.raises(ValueError, match="row_weight carries no gradient"):
        moe.sort_tokens(cfg, idx, w)
    for call in (lambda: moe.sort_tokens(cfg, idx, w.detach()), torch.no_grad()(lambda: moe.sort_tokens(cfg, idx, w))):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):  # what is wrong with them otherwise
            call()


@pytest.mark.gpu
def test_sorted_weights_without_a_graph_are_taken():
    cfg = moe.make_config(T=4, h=256, E=8, k=2, I=256)
    idx, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.rand(4, 2, device="cuda", requires_grad=True)
    want = w.detach().flatten()
    assert torch.equal(moe.sort_tokens(cfg, idx, w.detach())["row_weight"], want)
    with torch.no_grad():
        assert torch.equal(moe.sort_tokens(cfg, idx, w)["row_weight"], want)
