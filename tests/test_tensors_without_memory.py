"""Tensors that have a shape and a device but no memory of their own (of a wrapper's class, or with a storage that was given
up): refused, also where the argument may be left out, and before any CUDA call."""
import pytest
import torch

from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe


class Wrapper(torch.Tensor):
    """What a wrapper's class looks like from outside: all but the memory."""

    @staticmethod
    def __new__(cls, like, offset=0):
        strides = [1] if like.dim() == 1 else [like.shape[1], 1]
        return torch.Tensor._make_wrapper_subclass(cls, like.shape, strides=strides, dtype=like.dtype, device="cuda:0",
                                                   storage_offset=offset)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise RuntimeError(str(func))


def given_up(t):
    t = t.clone()
    t.untyped_storage().resize_(0)
    return t


def given_up_slice(t):
    t = torch.cat((t, t))[t.shape[0]:]
    t.untyped_storage().resize_(0)
    return t


KINDS = {"wrapper": Wrapper, "wrapper with an offset": lambda t: Wrapper(t, 64), "given up": given_up,
         "given up, a slice": given_up_slice}


def calls(make, device):
    """A call for every tensor that a call takes, in its place what make() makes of it."""
    cfg = moe.make_config(T=4, h=256, E=8, k=2, I=256)
    x, w, tw = torch.randn(4, 16, device=device), torch.ones(16, device=device), torch.ones(4, 2, device=device)
    idx = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device=device)
    off = torch.arange(9, dtype=torch.int32, device=device)
    z, yd, q = torch.randn(4, 8, device=device), torch.randn(8, 16, device=device), torch.zeros(4, 16, dtype=torch.uint8, device=device)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=device)
    s = torch.ones(4, 1, device=device)
    for f, args in ((moe.rms_norm, (x, w, x)), (moe.rms_norm_fp8, (x, w, x)), (moe.rms_norm_backward, (x, x, w, 1e-6, x, True, ws)),
                    (moe.sort_tokens, (cfg, idx, tw, ws)), (moe.permute, (cfg, q, idx, off, s)),
                    (moe.unpermute, (cfg, yd, idx, tw, x)), (moe.unpermute_backward, (cfg, x, yd, idx, off, tw)),
                    (moe.route_weights, (cfg, z)), (moe.route_backward, (cfg, z, idx, tw))):
        for i, a in enumerate(args):
            if isinstance(a, torch.Tensor):
                yield f"{f.__name__} {i}", lambda: f(*args[:i], make(a), *args[i + 1:])


def check(device):
    pkg_build.build()
    moe.load()
    for kind, make in KINDS.items():
        for name, call in calls(make, device):
            before = moe.launch_count()
            with pytest.raises(ValueError, match="memory"):
                call()
            assert moe.launch_count() == before, (kind, name)


def test_refused_on_the_host():
    """The other arguments are CPU tensors here: what is asked first is whether there is memory."""
    check("cpu")


def test_weights_and_optional_addresses():
    t = torch.ones(8)
    for make in KINDS.values():
        for f in (lambda: moe._ptr(make(t)), lambda: moe._address(make(t)), lambda: moe.Weights(t, bias=make(t))):
            with pytest.raises(ValueError, match="memory"):
                f()
    empty = torch.empty(0)
    assert moe._ptr(None) is None and moe._address(None) is None and moe._address(empty) == empty.data_ptr()
    assert moe._address(t) == t.data_ptr() and moe._address(torch.nn.Parameter(t)) == t.data_ptr()


@pytest.mark.gpu
def test_refused_on_the_gpu():
    check("cuda")


@pytest.mark.gpu
def test_tensors_without_elements_are_taken():
    cfg = moe.make_config(T=0, h=256, E=8, k=2, I=256)
    s = moe.sort_tokens(cfg, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    x = torch.empty(0, 16, device="cuda")
    assert moe.rms_norm(x, torch.ones(16, device="cuda"), x)[0].shape == (0, 16)
    assert moe.unpermute(cfg, x, s["inv_pos"], torch.empty(0, 2, device="cuda"), x).shape == (0, 16)
