"""Narrow rows that share a warp, at the widths where their lanes change: the norm, the rows by expert and back, and the
gradients, with what lies beside a row (a NaN, an infinity, a row that is not there) and numbers of rows that leave a warp
partly empty. Tolerances as in test_gpu_rms_norm.py and test_gpu_permute.py: a lane's additions are at most 8 here."""
import itertools

import pytest
import torch

import plain_rows as plain
import routing_dispatch_expert_gb300 as rde
from plain_rows import HALF, TINY, U32
from routing_dispatch_expert_gb300 import build as pkg_build
from test_gpu_permute import choices, config
from test_gpu_rms_norm import EPS, check_codes, check_gradient, check_total_and_y, close, rows

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
COLS = [2, 5, 9, 31, 32, 33, 36, 63, 65, 100, 127]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind,other", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_norm(cols, kind, other):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    w = 1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")
    for n, ld in itertools.product((1, 2, 63, 66, 517), (cols, cols + 3)):
        x, r = rows(gen, n, ld, kind)[:, :cols], rows(gen, n, ld, other, 3.0)[:, :cols]
        want_y, want_t = plain.norm(x, w, r, EPS)
        out = rde.rms_norm_fp8(x, w, r, EPS, with_y=True)
        check_total_and_y(out["y"], out["total"], want_y, want_t, kind, other)
        check_codes(out["q"], out["s"], want_y, cols)
        y, total = rde.rms_norm(x, w, r, EPS)
        assert torch.equal(y, out["y"]) and torch.equal(total, out["total"])


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind,other", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_norm_gradient(cols, kind, other):
    gen = torch.Generator(device="cuda").manual_seed(cols + 200)
    for n, ld, wkind in itertools.product((1, 2, 63, 66, 5003), (cols, cols + 3), (None, F32)):
        dy, t = rows(gen, n, cols, kind), rows(gen, n, ld, other, 2.0)[:, :cols]
        dt = rows(gen, n, cols, other) if n % 2 else None
        w = None if wkind is None else (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(wkind)
        check_gradient(dy, t, w, dt, rde.rms_norm_backward(dy, t, w, EPS, dt))


@pytest.mark.parametrize("cols", [5, 33, 64, 127])
def test_rows_beside_a_nan(cols):
    """A row's neighbours in its warp keep their numbers, whatever it holds."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dy = rows(gen, 41, cols, BF16), rows(gen, 41, cols, BF16)
    y, dx = rde.rms_norm(x, eps=EPS), rde.rms_norm_backward(dy, x, None, EPS)[0]
    q = rde.rms_norm_fp8(x, eps=EPS)
    for value in (float("nan"), float("inf")):
        bad = x.clone()
        bad[7::9, cols - 1] = value
        keep = torch.isfinite(bad.float()).all(1)
        assert torch.equal(rde.rms_norm(bad, eps=EPS)[keep], y[keep])
        assert torch.equal(rde.rms_norm_backward(dy, bad, None, EPS)[0][keep], dx[keep])
        got = rde.rms_norm_fp8(bad, eps=EPS)
        assert torch.equal(got["q"][keep], q["q"][keep]) and torch.equal(got["s"][keep], q["s"][keep])
        # tokens beside each other in the rows' way back
        cfg = config(41, 4, 1)
        s = rde.sort_tokens(cfg, choices(41, 4, 1, seed=2))
        back = rde.unpermute(cfg, rde.permute(cfg, bad, s["inv_pos"], s["offsets"]), s["inv_pos"])
        assert torch.equal(back[keep], bad[keep])
        dw = rde.unpermute_backward(cfg, dy, rde.permute(cfg, bad, s["inv_pos"], s["offsets"]), s["inv_pos"], s["offsets"])[1]
        assert torch.isfinite(dw[keep]).all() and not torch.isfinite(dw[~keep]).any()


@pytest.mark.parametrize("T,k", [(1, 1), (3, 2), (67, 3), (130, 4), (514, 5), (35, 9)])
@pytest.mark.parametrize("kind", [F32, BF16, F16])
def test_rows_and_back(T, k, kind):
    E = 12
    cfg = config(T, E, k, capacity_factor=1.5)
    s = rde.sort_tokens(cfg, choices(T, E, k, seed=T, pad=0.3))
    inv, token, n_held = s["inv_pos"], s["row_token"].long(), int(s["offsets"][-1])
    for cols in COLS:
        gen = torch.Generator(device="cuda").manual_seed(cols)
        x, dy, base = (rows(gen, T, cols, kind) for _ in range(3))
        yd = rows(gen, T * k, cols, kind)
        yd[n_held:] = float("nan")  # rows that hold nothing are not read
        w = torch.rand(T, k, generator=gen, device="cuda")
        xd = rde.permute(cfg, x, inv, s["offsets"])
        assert torch.equal(xd, torch.where((token >= 0).unsqueeze(1), x[token.clamp(min=0)], torch.zeros((), dtype=kind, device="cuda")))
        y, size = plain.unpermute(yd, inv, w, base)
        close(rde.unpermute(cfg, yd, inv, w, base), y, (k + 2) * U32 * size + HALF[kind] * y.abs() * (1 + 2.0 ** -8) + TINY[kind], "y")
        dyd, dw, size = plain.unpermute_backward(dy, yd, inv, w)
        got = rde.unpermute_backward(cfg, dy, yd, inv, s["offsets"], w)
        close(got[0], dyd, (HALF[kind] + 2 * U32) * dyd.abs() + TINY[kind], "dyd")
        assert (got[0][n_held:] == 0).all() and (got[1][inv < 0] == 0).all()
        close(got[1], dw, 14 * U32 * size, "dweights")


@pytest.mark.parametrize("cols", [1, 16, 33, 64, 65, 100, 129, 200, 240, 256, 257, 300, 511, 1000, 1024, 1040, 2047])
def test_codes_by_expert(cols):
    """8-bit rows and their scales at the widths where the words of a lane change."""
    for T, k, pad in ((1, 1, 0.0), (45, 3, 0.2), (700, 8, 0.5), (60, 2, 1.0)):
        cfg = config(T, 12, k)
        s = rde.sort_tokens(cfg, choices(T, 12, k, seed=T, pad=pad))
        token = s["row_token"].long()
        held = (token >= 0).unsqueeze(1)
        x = torch.randint(1, 255, (T, cols), dtype=torch.uint8, device="cuda")
        scales = torch.rand(T, (cols + 127) // 128, device="cuda")
        q, qs = rde.permute(cfg, x, s["inv_pos"], s["offsets"], scales)
        assert torch.equal(q, torch.where(held, x[token.clamp(min=0)], torch.zeros((), dtype=torch.uint8, device="cuda")))
        assert torch.equal(qs, torch.where(held, scales[token.clamp(min=0)], 0.0))
        assert torch.equal(q, rde.permute(cfg, x, s["inv_pos"], s["offsets"]))


EVEN = [130, 250, 258, 1002, 2050, 4102, 16382]


@pytest.mark.parametrize("cols", EVEN)
@pytest.mark.parametrize("kind,other", [(BF16, BF16), (F16, F32)])
def test_norm_of_even_rows(cols, kind, other):
    """16-bit rows of an even number of columns that are not whole 16 bytes, whose begins lie an even or an odd number apart."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    for n, more, wkind in itertools.product((1, 2, 35, 311), (0, 2, 3), (None, kind, F32)):
        if n == 311 and cols > 4102:
            continue
        w = None if wkind is None else (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(wkind)
        x, r = rows(gen, n, cols + more, kind)[:, :cols], rows(gen, n, cols + more, other, 3.0)[:, :cols]
        want_y, want_t = plain.norm(x, w, r, EPS)
        out = rde.rms_norm_fp8(x, w, r, EPS, with_y=True)
        check_total_and_y(out["y"], out["total"], want_y, want_t, kind, other)
        check_codes(out["q"], out["s"], want_y, cols)
        dy, dt = rows(gen, n, cols, kind), rows(gen, n, cols, other) if n % 2 else None
        check_gradient(dy, r, w, dt, rde.rms_norm_backward(dy, r, w, EPS, dt))


@pytest.mark.parametrize("cols", EVEN[:-1])
@pytest.mark.parametrize("kind", [BF16, F16])
def test_even_rows_and_back(cols, kind):
    for T, k in ((1, 1), (67, 2), (130, 4), (300, 8), (35, 11)):
        cfg = config(T, 16, k, capacity_factor=1.5)
        s = rde.sort_tokens(cfg, choices(T, 16, k, seed=T, pad=0.2))
        inv, n_held = s["inv_pos"], int(s["offsets"][-1])
        gen = torch.Generator(device="cuda").manual_seed(cols)
        dy, base = (rows(gen, T, cols, kind) for _ in range(2))
        yd = rows(gen, T * k, cols, kind)
        yd[n_held:] = float("nan")
        w = torch.rand(T, k, generator=gen, device="cuda")
        y, size = plain.unpermute(yd, inv, w, base)
        close(rde.unpermute(cfg, yd, inv, w, base), y, (k + 2) * U32 * size + HALF[kind] * y.abs() * (1 + 2.0 ** -8) + TINY[kind], "y")
        dyd, dw, size = plain.unpermute_backward(dy, yd, inv, w)
        got = rde.unpermute_backward(cfg, dy, yd, inv, s["offsets"], w)
        close(got[0], dyd, (HALF[kind] + 2 * U32) * dyd.abs() + TINY[kind], "dyd")
        assert (got[0][n_held:] == 0).all() and (got[1][inv < 0] == 0).all()
        close(got[1], dw, (8 * (cols // 256 + 1) + 14) * U32 * size, "dweights")
