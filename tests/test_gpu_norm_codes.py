"""The norm's 8-bit codes are those of the FP8 layer's rows: e4m3 of the correctly rounded quotient of y and its scale.

With x of ones, eps 0 and a weight, the mean of the squares is 1 exactly and y is the weight exactly, so the codes can be said
bit by bit: equal, without a tolerance. The weights are chosen next to the midpoints of two codes, where the quotient's last bit
decides."""
import numpy as np
import pytest
import torch

import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build

pytestmark = pytest.mark.gpu
F32, BF16, F16, U8 = torch.float32, torch.bfloat16, torch.float16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def midpoints():
    """The numbers halfway between two neighbouring e4m3 values."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    return (v[1:] + v[:-1]) / np.float32(2)


def near_midpoints(cols, seed):
    """fp32 [cols]: in each block of 128 a largest magnitude of its own, and numbers whose quotient by the block's scale is
    within a step of a midpoint of two codes; zeros of both signs."""
    rng = np.random.default_rng(seed)
    out = np.zeros(cols, np.float32)
    mid = midpoints()
    for c0 in range(0, cols, 128):
        n = min(128, cols - c0)
        amax = np.float32(np.exp2(rng.uniform(-20, 20)))
        scale = amax / np.float32(448)
        v = rng.choice(mid, n).astype(np.float32) * scale * rng.choice(np.float32([-1, 1]), n)
        v = np.nextafter(v, v * rng.choice(np.float32([0.5, 1, 2]), n)).astype(np.float32)  # down, as it is, or up
        v[rng.integers(n)] = amax
        if n > 8:
            zero = rng.choice(np.flatnonzero(np.abs(v) < amax), 2, replace=False)
            v[zero] = np.float32([0.0, -0.0])
        out[c0:c0 + n] = v
    return out


def codes_and_scales(v):
    """By the definition, in fp32 arithmetic on the host."""
    cols, n = v.size, -(-v.size // 128)
    s = np.array([np.abs(v[128 * b:128 * b + 128]).max() for b in range(n)], np.float32) / np.float32(448)
    q = v / np.repeat(s, 128)[:cols]
    assert q.dtype == np.float32
    return torch.from_numpy(q).clamp(-448, 448).to(torch.float8_e4m3fn).view(U8), torch.from_numpy(s)


@pytest.mark.parametrize("cols", [1, 8, 33, 34, 64, 72, 128, 129, 256, 1000, 1003, 4096, 7168, 16384])
@pytest.mark.parametrize("kind", [BF16, F16, F32])
@pytest.mark.parametrize("other", [None, F32])
def test_codes_are_those_of_the_quotient(cols, kind, other):
    for seed in range(6):
        v = near_midpoints(cols, seed)
        q, s = codes_and_scales(v)
        x = torch.ones(3, cols, device="cuda", dtype=kind)
        r = None if other is None else torch.zeros(3, cols, device="cuda", dtype=other)
        x[1] = -1
        out = rde.rms_norm_fp8(x, torch.from_numpy(v).cuda(), r, eps=0.0)
        assert torch.equal(out["s"].cpu(), s.expand(3, -1))
        got = out["q"].cpu()
        for row, sign in ((0, 0), (1, 128), (2, 0)):
            assert torch.equal(got[row], q ^ sign), f"{int((got[row] != q ^ sign).sum())} codes of {cols}"


@pytest.mark.parametrize("scale_exponent", [-126, -100, 60, 99])
def test_extreme_scales(scale_exponent):
    """Scales from the least one up to where the lower part of 1 / scale is no normal number any more."""
    v = near_midpoints(2048, 3)
    blocks = v.reshape(-1, 128)
    blocks *= (np.exp2(np.float64(scale_exponent)) * 448 / np.abs(blocks).max(1, keepdims=True)).astype(np.float32)
    v = blocks.reshape(-1)
    q, s = codes_and_scales(v)
    out = rde.rms_norm_fp8(torch.ones(1, 2048, device="cuda"), torch.from_numpy(v).cuda(), eps=0.0)
    if scale_exponent == -126:
        s = s.clamp(min=2.0 ** -126)
        q = torch.from_numpy(v / np.repeat(s.numpy(), 128)).clamp(-448, 448).to(torch.float8_e4m3fn).view(U8)
    assert torch.equal(out["s"].cpu(), s.view(1, -1)) and torch.equal(out["q"].cpu(), q.view(1, -1))


def test_rows_as_the_fp8_layer_quantises_them():
    T, h = 8, 2048
    w = torch.stack([torch.from_numpy(near_midpoints(h, 10 + t)) for t in range(T)]).cuda().to(BF16)
    cfg = rde.make_config(T=T, h=h, E=1, k=1, I=256, dtype="fp8")
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    xd = torch.empty(T, h, dtype=U8, device="cuda")
    xs = torch.empty(T, h // 128, device="cuda")
    ws = rde.alloc_workspace(cfg)
    rde.device_status(cfg, ws)
    rde.dispatch(cfg, w, torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda"), i32(1), i32(2),
                 i32(T, 1), i32(T), torch.empty(T, device="cuda"), xd, xs, ws)
    for t in range(T):
        out = rde.rms_norm_fp8(torch.ones(1, h, dtype=BF16, device="cuda"), w[t], eps=0.0)
        assert torch.equal(out["q"][0], xd[t]) and torch.equal(out["s"][0], xs[t])
