"""The norm, its 8-bit output and its gradient on the GPU, against the definition in 64 bits.

Tolerances, with u = 2^-24: the sum of squares of a row passes through at most 16 fused additions of a lane, 5 of a warp and 5
of a block (all terms positive: relative error 27 u with the squares' own), the division, eps and root add 3 u and half of
the sum's error, and y = t * rstd * w two roundings more: below 20 u in all; 32 u is allowed. The half step of the output's type
comes on top."""
import itertools

import pytest
import torch

import plain_rows as plain
import routing_dispatch_expert_gb300 as rde
from plain_rows import HALF, TINY, U32
from routing_dispatch_expert_gb300 import build as pkg_build

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5
COLS = [1, 7, 8, 24, 40, 64, 72, 128, 129, 136, 255, 256, 257, 1000, 2048, 2049, 2304, 4101, 7168, 8192, 8200, 16383, 16384]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def rows(gen, n, cols, dtype, scale=1.0):
    return (torch.randn(n, cols, generator=gen, device="cuda") * scale).to(dtype)


def close(got, want, bound, name):
    """|got - want| <= bound, all in 64 bits."""
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), f"{name}: {float(off.max())} over the bound at {int(off.argmax())}"


def check_total_and_y(y, total, want_y, want_t, kind, other):
    close(y, want_y, (HALF[kind] + 32 * U32) * (1 + HALF[kind]) * want_y.abs() + TINY[kind], "y")
    if total is not None:
        close(total, want_t, (HALF[other] + U32) * (1 + U32) * want_t.abs() + TINY[other], "total")


def check_codes(q, s, y, cols):
    n = (cols + 127) // 128
    big = torch.zeros(y.shape[0], 128 * n, dtype=torch.float64, device=y.device)
    big[:, :cols] = y
    scale = big.view(-1, n, 128).abs().amax(-1) / 448
    scale = torch.where(scale == 0, 1.0, scale.clamp(min=2.0 ** -126))
    close(s, scale, 34 * U32 * scale, "scale")  # the division's own on top of y's
    value = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :cols]
    step = s.double().repeat_interleave(128, 1)[:, :cols] * 2.0 ** -10  # half the least code
    # half a step of the code, at most 2^-4 of the value, the errors of y and scale, and of the quotient
    close(value, y, 2.0 ** -4 * y.abs() * (1 + 2.0 ** -10) + step + 72 * U32 * y.abs(), "codes")


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", [BF16, F16, F32])
def test_norm(cols, kind):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    for n, other, wkind in itertools.product([1, 19], {None, kind, F32}, {None, kind, F32}):
        x = rows(gen, n, cols, kind)
        r = None if other is None else rows(gen, n, cols, other, 3.0)
        w = None if wkind is None else (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(wkind)
        want_y, want_t = plain.norm(x, w, r, EPS)
        got = rde.rms_norm(x, w, r, EPS)
        y, total = got if r is not None else (got, None)
        check_total_and_y(y, total, want_y, want_t, kind, other)
        out = rde.rms_norm_fp8(x, w, r, EPS, with_y=True)
        assert torch.equal(out["y"], y) and (r is None) == ("total" not in out)
        assert r is None or torch.equal(out["total"], total)
        check_codes(out["q"], out["s"], want_y, cols)
        only = rde.rms_norm_fp8(x, w, r, EPS)
        assert "y" not in only and torch.equal(only["q"], out["q"]) and torch.equal(only["s"], out["s"])


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("ld", [264, 259, 512])
def test_strided_rows(kind, ld):
    """Rows that lie apart, on 16 bytes and not; a row that is a view of one, and the rows between are not touched."""
    gen = torch.Generator(device="cuda").manual_seed(ld)
    for cols in (250, 256):
        x, r = rows(gen, 33, ld, kind)[:, :cols], rows(gen, 33, ld, kind)[:, :cols]
        want_y, want_t = plain.norm(x, None, r, EPS)
        y, total = rde.rms_norm(x, None, r, EPS)
        check_total_and_y(y, total, want_y, want_t, kind, kind)
        out = rde.rms_norm_fp8(x, None, None, EPS)
        check_codes(out["q"], out["s"], plain.norm(x, None, None, EPS)[0], cols)
        w = torch.ones(cols, device="cuda")
        dy = r.contiguous()
        check_gradient(dy, x, w, None, rde.rms_norm_backward(dy, x, w, EPS))


def test_special_values():
    x = torch.randn(6, 384, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e-30
    x[5, :128] = 0
    y = rde.rms_norm(x, None, eps=1e-6)
    out = rde.rms_norm_fp8(x, None, eps=1e-6, with_y=True)
    assert (y[1] == 0).all() and y[2].isnan().all() and y[3, 7].isnan() and (y[3, 8:] == 0).all()
    values = out["q"].view(torch.float8_e4m3fn).float() * out["s"].repeat_interleave(128, 1)
    assert (out["s"][1] == 1).all() and (values[1] == 0).all()
    assert values[2].isnan().all() and values[3, :128].isnan().all()  # never a finite number made of an infinity
    assert out["s"][5, 0] == 1 and (values[5, :128] == 0).all()
    tiny = rde.rms_norm_fp8(x[4:5], torch.full((384,), 1e-12, device="cuda"), eps=1e-6)  # y far below 448 * 2^-126
    assert (tiny["s"] == 2.0 ** -126).all()
    check_codes(tiny["q"], tiny["s"], plain.norm(x[4:5], torch.full((384,), 1e-12, device="cuda"), None, 1e-6)[0], 384)
    assert torch.isfinite(rde.rms_norm_backward(x[:2], x[:2], None, 1e-6)[0]).all()


def test_no_rows_and_refusals():
    x = torch.empty(0, 64, device="cuda", dtype=BF16)
    w = torch.ones(64, device="cuda", dtype=BF16)
    assert rde.rms_norm(x, w).shape == (0, 64)
    dx, _, dw = rde.rms_norm_backward(x, x, w)
    assert dx.shape == (0, 64) and (dw == 0).all()
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(rde.MoeError, match="16384"):
        rde.rms_norm(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(ValueError, match="weight must have shape"):
        rde.rms_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="residual must be"):
        rde.rms_norm(x.to(BF16), residual=x.half())
    with pytest.raises(ValueError, match="elements of a row of x must be contiguous"):
        rde.rms_norm(x.t())
    with pytest.raises(ValueError, match="dy must be contiguous"):
        rde.rms_norm_backward(x[:, :32], x[:, :32])
    with pytest.raises(rde.MoeError, match="16-byte aligned"):
        rde.rms_norm(x.flatten()[1:65].view(1, 64))
    with pytest.raises(rde.MoeError, match="too small"):
        rde.rms_norm_backward(x, x, torch.ones(64, device="cuda"), ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------------------------
# the gradient
# ------------------------------------------------------------------------------------------
def check_gradient(dy, t, w, dt, got):
    """Errors relative to sums of magnitudes: the two sums of a row as above (32 u, the second one of terms of any sign),
    their product and the four roundings behind them, 80 u in all; a column's sum over the rows passes through at most
    ceil(rows / 152) + 8 additions of a block, ceil(blocks / 32) of a lane and 5 of a warp, each u, on terms that are 40 u off."""
    dx, dr, dw = got
    d, want_dw, size, dw_size = plain.norm_backward(dy, t, w, EPS, dt)
    close(dx, d, 80 * U32 * size + HALF[dx.dtype] * d.abs() * (1 + 2.0 ** -8) + TINY[dx.dtype], "dx")
    close(dr, d, 80 * U32 * size + HALF[dr.dtype] * d.abs() * (1 + 2.0 ** -8) + TINY[dr.dtype], "dresidual")
    if w is not None:
        n = dy.shape[0] // 152 + 1 + 8 + 152 + 5 + 40
        close(dw, want_dw, n * U32 * dw_size + HALF[dw.dtype] * want_dw.abs() * (1 + 2.0 ** -8) + TINY[dw.dtype], "dweight")
    else:
        assert dw is None


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", [BF16, F16, F32])
def test_gradient(cols, kind):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    for n, other, wkind, more in itertools.product([1, 21, 700], {kind, F32}, {None, kind, F32}, [False, True]):
        if n == 700 and (cols > 4101 or wkind is kind):
            continue
        dy, t = rows(gen, n, cols, kind), rows(gen, n, cols, other, 2.0)
        dt = rows(gen, n, cols, other) if more else None
        w = None if wkind is None else (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(wkind)
        check_gradient(dy, t, w, dt, rde.rms_norm_backward(dy, t, w, EPS, dt))


def test_gradient_of_many_rows():
    gen = torch.Generator(device="cuda").manual_seed(5)
    for n, cols, kind in ((20001, 64, F32), (70000, 8, BF16), (70001, 33, BF16), (30011, 128, F16), (5003, 520, F16), (3000, 7168, BF16),
                          (2001, 4101, F32), (2001, 2051, BF16)):
        dy, t, w = rows(gen, n, cols, kind), rows(gen, n, cols, kind), torch.randn(cols, generator=gen, device="cuda")
        got = rde.rms_norm_backward(dy, t, w, EPS)
        check_gradient(dy, t, w, None, got)
        again = rde.rms_norm_backward(dy, t, w, EPS)
        assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits


def test_gradient_is_the_norms_by_differences():
    """Differences of the kernel's own output, fp32: a step of 2^-6 of inputs of size 1 leaves h^2 / 6 times a third
    derivative (of about the size of dy) and 2^-24 * 40 of |y| / h: 1e-3 of the gradient's scale allowed."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, w, dy = rows(gen, 1, 48, F32), 1 + rows(gen, 1, 48, F32)[0] * 0.1, rows(gen, 1, 48, F32)
    dx, _, dw = rde.rms_norm_backward(dy, x, w, EPS)
    h = 2.0 ** -6
    for v, d, f in ((x, dx[0], lambda e: rde.rms_norm(x + e, w, eps=EPS)), (w, dw, lambda e: rde.rms_norm(x, w + e[0], eps=EPS))):
        for i in range(0, 48, 5):
            e = torch.zeros(1, 48, device="cuda")
            e[0, i] = h
            got = float(((f(e) - f(-e)).double() * dy.double()).sum()) / (2 * h)
            assert abs(got - float(d[i])) < 1e-3 * float(dy.abs().max())


@pytest.mark.parametrize("kind,other", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_autograd(kind, other):
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, r = rows(gen, 9, 384, kind).requires_grad_(), rows(gen, 9, 384, other).requires_grad_()
    w = torch.randn(384, generator=gen, device="cuda").requires_grad_()
    dy, dt = rows(gen, 9, 384, kind), rows(gen, 9, 384, other)
    y, total = rde.rms_norm(x, w, r, EPS)
    torch.autograd.backward((y, total), (dy, dt))
    dx, dr, dw = rde.rms_norm_backward(dy, total.detach(), w.detach(), EPS, dt)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dr) and torch.equal(w.grad, dw)
    assert x.grad.dtype == kind and r.grad.dtype == other
    x.grad = r.grad = w.grad = None
    out = rde.rms_norm_fp8(x, w, r, EPS, with_y=True)  # codes carry no gradient, y does
    assert not out["q"].requires_grad and not out["s"].requires_grad
    (out["y"].float() * dy.float()).sum().backward()
    dx, dr, dw = rde.rms_norm_backward(dy, total.detach(), w.detach(), EPS)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dr) and torch.equal(w.grad, dw)
    x.grad = r.grad = w.grad = None
    rde.rms_norm(x, w, r, EPS)[1].sum().backward()  # the total alone: a sum, and an expanded gradient
    assert (x.grad == 1).all() and (r.grad == 1).all() and w.grad is None
    x.grad = None
    rde.rms_norm(x, None, eps=EPS).sum().backward()
    assert torch.equal(x.grad, rde.rms_norm_backward(torch.ones_like(x), x.detach(), None, EPS)[0])
    with torch.no_grad():
        assert not rde.rms_norm(x, w, eps=EPS).requires_grad


def test_autograd_guards():
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    d, = torch.autograd.grad(rde.rms_norm(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()
    z = x * 1.0
    y = rde.rms_norm(z)
    z.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
