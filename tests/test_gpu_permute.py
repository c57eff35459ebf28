"""Sort, rows into expert order and back, and their gradients on the GPU: the sort and the copies equal to the definition,
sums within the roundings of fp32 (u = 2^-24 for each addition a term passes through) and one of the output's type."""
import math

import numpy as np
import pytest
import torch

import plain_rows as plain
import routing_dispatch_expert_gb300 as rde
from plain_rows import HALF, TINY, U32
from routing_dispatch_expert_gb300 import build as pkg_build
from test_gpu_rms_norm import close

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def config(T, E, k, **kw):
    return rde.make_config(T=T, h=256, E=E, k=k, I=256, **kw)


def choices(T, E, k, seed=0, pad=0.0, skew=1.0, twice=False):
    """Chosen experts, some liked more; padded tokens, and with `twice` repeated and out-of-range ones."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, E, generator=gen, device="cuda") + skew * torch.randn(E, generator=gen, device="cuda")
    idx = torch.topk(z, k).indices.int()
    if twice:
        idx = torch.randint(-1, E + 1, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    return torch.where(torch.rand(T, 1, generator=gen, device="cuda") < pad, -1, idx).int().contiguous()


def check_sort(cfg, idx, capacity=None, placement=None):
    w = torch.rand(cfg.T, cfg.k, device="cuda") + 0.1
    got = rde.sort_tokens(cfg, idx, w)
    want = plain.sort(idx.cpu(), cfg.E, capacity, placement)
    for name in ("counts", "offsets", "row_token"):
        assert got[name].tolist() == want[name], name
    assert got["inv_pos"].flatten().tolist() == want["inv_pos"]
    source = torch.tensor(want["source"], device="cuda", dtype=torch.long)
    assert torch.equal(got["row_weight"], torch.where(source >= 0, w.flatten()[source.clamp(min=0)], 0.0))
    plainly = rde.sort_tokens(cfg, idx)
    assert "row_weight" not in plainly and torch.equal(plainly["inv_pos"], got["inv_pos"])
    return got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (31, 3, 2), (256, 256, 8), (257, 256, 8), (1000, 60, 6), (2048, 8, 1),
                                   (2049, 8, 1), (700, 1024, 3), (513, 40, 32), (16384, 256, 8)])
@pytest.mark.parametrize("pad", [0.0, 0.3, 1.0])
def test_sort(T, E, k, pad):
    check_sort(config(T, E, k), choices(T, E, k, seed=T, pad=pad))


@pytest.mark.parametrize("T,E,k", [(40, 3, 3), (5000, 12, 4)])
def test_sort_repeated_and_out_of_range(T, E, k):
    check_sort(config(T, E, k), choices(T, E, k, seed=1, twice=True))
    check_sort(config(T, E, k), torch.full((T, k), E - 1, device="cuda", dtype=torch.int32))  # all to one expert


@pytest.mark.parametrize("T,E,k,factor", [(999, 60, 6, 1.25), (50, 4, 2, 0.1), (4000, 16, 2, 1.0)])
def test_sort_with_a_capacity(T, E, k, factor):
    cfg = config(T, E, k, capacity_factor=factor)
    check_sort(cfg, choices(T, E, k, seed=2, pad=0.1), math.ceil(np.float32(factor) * T * k / E))
    check_sort(cfg, choices(T, E, k, seed=2, twice=True), math.ceil(np.float32(factor) * T * k / E))


@pytest.mark.parametrize("T,factor", [(100, 0.0), (3000, 0.0), (3000, 1.25)])
def test_sort_under_a_placement(T, factor):
    E, k = 16, 4
    idx = choices(T, E, k, seed=3, skew=2.0)
    load = torch.bincount(idx.flatten().long(), minlength=E).cpu().numpy()
    plan = rde.eplb_plan(load, 4, 8)
    cfg = config(T, E, k, capacity_factor=factor, placement=rde.Placement(plan))
    cap = math.ceil(np.float32(factor) * T * k / E) if factor else None
    got = check_sort(cfg, idx, cap, {n: plan[n].tolist() for n in ("slot_expert", "slot_replica", "replicas")})
    x = torch.randn(T, 32, device="cuda")
    xd = rde.permute(cfg, x, got["inv_pos"], got["offsets"])
    assert torch.equal(xd[got["inv_pos"][got["inv_pos"] >= 0].long()], x.repeat_interleave(k, 0)[got["inv_pos"].flatten() >= 0])


def test_sort_of_more_than_one_round_a_block():
    """Over 128 blocks' worth of 2048 assignments: blocks take several rounds. numpy's stable sort says the rest."""
    T, E, k = 70000, 33, 8
    idx = choices(T, E, k, seed=4, pad=0.05)
    got = rde.sort_tokens(config(T, E, k), idx)
    flat = idx.flatten().cpu().numpy()
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:(flat >= 0).sum()]
    inv = np.full(T * k, -1, np.int32)
    inv[order] = np.arange(order.size, dtype=np.int32)
    np.testing.assert_array_equal(got["inv_pos"].flatten().cpu().numpy(), inv)
    np.testing.assert_array_equal(got["row_token"].cpu().numpy()[:order.size], order // k)
    assert (got["row_token"][order.size:] == -1).all() and int(got["offsets"][-1]) == order.size


def test_sort_agrees_with_dispatch():
    T, E, k, h = 900, 64, 4, 256
    cfg = rde.make_config(T=T, h=h, E=E, k=k, I=256)
    idx, w = choices(T, E, k, seed=5), torch.rand(T, k, device="cuda")
    x = torch.randn(T, h, device="cuda").to(BF16)
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    c, o, p, t, rw = i32(E), i32(E + 1), i32(T, k), i32(T * k), torch.empty(T * k, device="cuda")
    xd = torch.empty(T * k, h, dtype=BF16, device="cuda")
    ws = rde.alloc_workspace(cfg)
    rde.device_status(cfg, ws)
    rde.dispatch(cfg, x, idx, w, c, o, p, t, rw, xd, None, ws)
    s = rde.sort_tokens(cfg, idx, w)
    for a, b in ((c, "counts"), (o, "offsets"), (p, "inv_pos"), (t, "row_token"), (rw, "row_weight")):
        assert torch.equal(a, s[b]), b
    assert torch.equal(xd, rde.permute(cfg, x, s["inv_pos"], s["offsets"]))
    y = torch.empty_like(x)
    rde.combine(cfg, xd, p, y)
    assert torch.equal(y, rde.unpermute(cfg, xd, s["inv_pos"]))


# ------------------------------------------------------------------------------------------
# rows
# ------------------------------------------------------------------------------------------
SHAPES = [(1, 4, 1), (77, 8, 2), (300, 33, 8), (130, 40, 17), (20, 64, 32)]
WIDTHS = [1, 2, 3, 8, 24, 33, 64, 72, 128, 255, 256, 1003, 4096, 4104]


def sorted_batch(T, E, k, pad=0.15, factor=1.25):
    cfg = config(T, E, k, capacity_factor=factor)
    return cfg, rde.sort_tokens(cfg, choices(T, E, k, seed=T + k, pad=pad))


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("cols", WIDTHS)
def test_permute(T, E, k, cols):
    cfg, s = sorted_batch(T, E, k)
    token = s["row_token"].long()
    for kind in (F32, BF16, F16, torch.uint8):
        for ld in (cols, cols + 5, cols + 16):
            full = torch.randn(T, ld, device="cuda")
            x = (full.to(kind) if kind is not torch.uint8 else (full * 60).to(torch.int8).view(torch.uint8))[:, :cols]
            n = (cols + 127) // 128
            scales = torch.rand(T, n, device="cuda") if kind is torch.uint8 else None
            got = rde.permute(cfg, x, s["inv_pos"], s["offsets"], scales)
            xd = got if scales is None else got[0]
            held = (token >= 0).unsqueeze(1)
            assert torch.equal(xd, torch.where(held, x[token.clamp(min=0)], torch.zeros((), dtype=kind, device="cuda")))
            if scales is not None:
                assert torch.equal(got[1], torch.where(held, scales[token.clamp(min=0)], 0.0))


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind", [F32, BF16, F16])
def test_unpermute_and_gradient(T, E, k, kind):
    cfg, s = sorted_batch(T, E, k)
    inv, held = s["inv_pos"], int(s["offsets"][-1])
    for cols in WIDTHS:
        gen = torch.Generator(device="cuda").manual_seed(cols)
        yd = torch.randn(T * k, cols, generator=gen, device="cuda").to(kind)
        base, dy = (torch.randn(T, cols, generator=gen, device="cuda").to(kind) for _ in range(2))
        yd[held:] = float("nan")  # rows that hold nothing are not read
        weights = torch.rand(T, k, generator=gen, device="cuda")
        weights[inv < 0] = float("nan")
        for w in (None, weights):
            for b in (None, base):
                y, size = plain.unpermute(yd, inv, w, b)
                close(rde.unpermute(cfg, yd, inv, w, b), y, (k + 2) * U32 * size + HALF[kind] * y.abs() * (1 + 2.0 ** -8) + TINY[kind],
                      "y")
            dyd, dw, size = plain.unpermute_backward(dy, yd, inv, w)
            got = rde.unpermute_backward(cfg, dy, yd, inv, s["offsets"], w)
            close(got[0], dyd, (HALF[kind] + 2 * U32) * dyd.abs() + TINY[kind], "dyd")
            assert (got[0][held:] == 0).all()
            # a lane's additions (8 for each of its chunks), 5 of a warp, 8 of a block
            close(got[1], dw, (8 * (cols // 256 + 1) + 14) * U32 * size, "dweights")
            assert (got[1][inv < 0] == 0).all()
            none = rde.unpermute_backward(cfg, dy, None, inv, s["offsets"], w)
            assert none[1] is None and torch.equal(none[0], got[0])


def test_gradient_by_differences():
    """y is linear in yd and in the weights: a difference of the sum <y, dy> is the gradient up to fp32's roundings, 20 u of
    the sum of magnitudes over a step of 1."""
    cfg, s = sorted_batch(6, 4, 3, pad=0.0)
    inv = s["inv_pos"]
    yd, dy, w = torch.randn(18, 40, device="cuda"), torch.randn(6, 40, device="cuda"), torch.rand(6, 3, device="cuda")
    dyd, dw = rde.unpermute_backward(cfg, dy, yd, inv, s["offsets"], w)
    f = lambda yd, w: float((rde.unpermute(cfg, yd, inv, w).double() * dy.double()).sum())  # noqa: E731
    size = 40 * U32 * float((plain.unpermute(yd, inv, w, None)[1] * dy.abs().double()).sum() + 10 * dy.abs().sum())
    for i in range(18):
        e = torch.zeros_like(yd)
        e[i, 2 * i] = 1.0
        assert abs(f(yd + e, w) - f(yd, w) - float(dyd[i, 2 * i])) < size
    for i in range(18):
        e = torch.zeros_like(w)
        e.view(-1)[i] = 1.0
        assert abs(f(yd, w + e) - f(yd, w) - float(dw.view(-1)[i])) < size


def test_far_rows():
    """Rows past 2^31 bytes and 2^31 elements of the expert-major buffers."""
    T, E, k, cols = 70000, 8, 8, 4096
    cfg = config(T, E, k)
    s = rde.sort_tokens(cfg, choices(T, E, k, seed=9))
    assert T * k * cols > 2 ** 31
    x = torch.randn(T, cols, device="cuda").to(BF16)
    xd = rde.permute(cfg, x, s["inv_pos"], s["offsets"])
    token = s["row_token"].long()
    for lo in range(0, T * k, 56000):
        assert torch.equal(xd[lo:lo + 56000], x[token[lo:lo + 56000]])
    w = torch.full((T, k), 0.125, device="cuda")
    assert torch.equal(rde.unpermute(cfg, xd, s["inv_pos"], w), x)  # eight eighths of the same row: exact
    dyd, dw = rde.unpermute_backward(cfg, x, xd, s["inv_pos"], s["offsets"], w)
    for lo in range(0, T * k, 56000):
        assert torch.equal(dyd[lo:lo + 56000], xd[lo:lo + 56000] * 0.125)
    want = x.double().square().sum(1, keepdim=True)
    close(dw, want.expand(T, k), 160 * U32 * want, "dweights")


def test_positions_outside_the_rows_are_left_out():
    """The kernels look at every position before they use it."""
    cfg, s = sorted_batch(40, 4, 2, pad=0.0, factor=0.0)
    inv = s["inv_pos"].clone()
    inv[3, 0], inv[7, 1], inv[9, 0] = 80, 2 ** 31 - 1, -2 ** 31
    clean = torch.where((inv < 0) | (inv >= 80), -1, inv).int()
    for cols in (24, 100, 333, 512):
        x, yd, w = torch.randn(40, cols, device="cuda"), torch.randn(80, cols, device="cuda"), torch.rand(40, 2, device="cuda")
        rows = clean[clean >= 0].long()
        assert torch.equal(rde.permute(cfg, x, inv, s["offsets"])[rows], rde.permute(cfg, x, clean, s["offsets"])[rows])
        assert torch.equal(rde.unpermute(cfg, yd, inv, w), rde.unpermute(cfg, yd, clean, w))
        a, b = (rde.unpermute_backward(cfg, x, yd, i, s["offsets"], w) for i in (inv, clean))
        assert torch.equal(a[0][rows], b[0][rows]) and torch.equal(a[1], b[1])


def test_no_tokens_and_refusals():
    cfg = config(0, 4, 2)
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    s = rde.sort_tokens(cfg, idx, torch.empty(0, 2, device="cuda"))
    assert s["counts"].tolist() == [0] * 4 and s["offsets"].tolist() == [0] * 5
    x = torch.empty(0, 16, device="cuda")
    assert rde.permute(cfg, x, idx, s["offsets"]).shape == (0, 16)
    assert rde.unpermute(cfg, x, idx).shape == (0, 16)
    assert rde.unpermute_backward(cfg, x, x, idx, s["offsets"])[1].shape == (0, 2)
    cfg, s = sorted_batch(10, 4, 2)
    x = torch.zeros(10, 16, device="cuda")
    yd = torch.zeros(20, 16, device="cuda")
    for call, text in ((lambda: rde.permute(cfg, x[:9], s["inv_pos"], s["offsets"]), "x must have shape"),
                       (lambda: rde.permute(cfg, x, s["inv_pos"][:9], s["offsets"]), "inv_pos must have shape"),
                       (lambda: rde.permute(cfg, x, s["inv_pos"], s["counts"]), "offsets must have shape"),
                       (lambda: rde.permute(cfg, x, s["inv_pos"], s["offsets"], x), "x must be torch.uint8"),
                       (lambda: rde.permute(cfg, x.double(), s["inv_pos"], s["offsets"]), "x must be"),
                       (lambda: rde.unpermute(cfg, x, s["inv_pos"]), "yd must have shape"),
                       (lambda: rde.unpermute(cfg, yd, s["inv_pos"], weights=x), "weights must have shape"),
                       (lambda: rde.unpermute(cfg, yd, s["inv_pos"], base=yd), "base must have shape"),
                       (lambda: rde.unpermute(cfg, yd, s["inv_pos"], base=x.half()), "base must be"),
                       (lambda: rde.unpermute_backward(cfg, x, x, s["inv_pos"], s["offsets"]), "yd must have shape"),
                       (lambda: rde.sort_tokens(cfg, s["inv_pos"].long()), "topk_idx must be"),
                       (lambda: rde.sort_tokens(cfg, s["inv_pos"], x), "topk_w must have shape")):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(rde.MoeError, match="too small"):
        rde.sort_tokens(config(3000, 4, 2), choices(3000, 4, 2), ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(rde.MoeError, match="16-byte aligned"):
        rde.permute(config(1, 4, 2), torch.zeros(17, device="cuda")[1:].view(1, 16), s["inv_pos"][:1].clone(), s["offsets"])


def test_autograd():
    T, E, k, cols = 50, 6, 3, 40
    cfg, s = sorted_batch(T, E, k)
    x = torch.randn(T, cols, device="cuda", requires_grad=True)
    w = torch.rand(T, k, device="cuda", requires_grad=True)
    base = torch.randn(T, cols, device="cuda", requires_grad=True)
    xd = rde.permute(cfg, x, s["inv_pos"], s["offsets"])
    y = rde.unpermute(cfg, xd * 2, s["inv_pos"], w, base, s["offsets"])
    dy = torch.randn(T, cols, device="cuda")
    y.backward(dy)
    dyd, dw = rde.unpermute_backward(cfg, dy, (xd * 2).detach(), s["inv_pos"], s["offsets"], w.detach())
    assert torch.equal(w.grad, dw) and torch.equal(base.grad, dy)
    assert torch.equal(x.grad, rde.unpermute(cfg, dyd * 2, s["inv_pos"]))
    for need in range(1, 8):  # any of the inputs alone
        a = [v.detach().clone().requires_grad_(bool(need >> i & 1)) for i, v in enumerate((xd * 2, w, base))]
        rde.unpermute(cfg, a[0], s["inv_pos"], a[1], a[2], s["offsets"]).backward(dy)
        for v, want in zip(a, (dyd, dw, dy)):
            assert (v.grad is None) if not v.requires_grad else torch.equal(v.grad, want)
    a = xd.detach().requires_grad_()  # an expanded gradient, without weights and base
    rde.unpermute(cfg, a, s["inv_pos"], offsets=s["offsets"]).sum().backward()
    assert torch.equal(a.grad, (s["row_token"] >= 0).float().unsqueeze(1).expand_as(a))
    with pytest.raises(ValueError, match="needs offsets"):
        rde.unpermute(cfg, a, s["inv_pos"])
