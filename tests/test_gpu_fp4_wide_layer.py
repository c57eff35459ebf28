"""The layer with 4-bit rows at hidden sizes of several passes and items of the dispatch copy, and experts of real size."""
import pytest
import torch

import plain_fp4 as plain
import routing_dispatch_expert_gb300 as rde
from test_gpu_fp4 import (FORMATS, Experts, built, check_hidden, hidden_of, layer_reference, product_tolerance,  # noqa: F401
                          rng, run_ffn)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("h", [512, 768, 1024, 1280, 2304, 7168])
@pytest.mark.parametrize("T,k,shared", [(1, 1, 0), (37, 4, 1), (300, 8, 0)])
def test_dispatch_writes_the_quantisers_rows(fmt, h, T, k, shared):
    """Codes and scales of every row, over all of h, are those of quantize_fp4 on the token's row."""
    E = 16
    cfg = rde.make_config(T=T, h=h, E=E, k=k, I=256, I_shared=256 * shared, dtype=fmt)
    x = torch.randn(T, h, generator=rng(h + T), device="cuda")
    x = (x * torch.exp(torch.randn(1, h, generator=rng(5), device="cuda"))).to(torch.bfloat16)
    g = torch.tensor([8.0 / 2688], device="cuda") if fmt == "nvfp4" else None
    act = rde.Fp4Activations(g) if fmt == "nvfp4" else None
    idx = torch.rand(T, E, generator=rng(2), device="cuda").argsort(1)[:, :k].int().contiguous()
    w = torch.rand(T, k, generator=rng(3), device="cuda")
    R = T * k
    n = plain.BLOCK[fmt]
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, inv, rt, rw = i32(E), i32(E + 1), i32(T, k), i32(R), torch.empty(R, device="cuda")
    xq = torch.zeros(R + T * shared, h // 2, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(R + T * shared, h // n, dtype=torch.uint8, device="cuda")
    ws = rde.alloc_workspace(cfg)
    rde.device_status(cfg, ws)
    rde.dispatch_fp4(cfg, act, x, idx, w, counts, offsets, inv, rt, rw, xq, xs, ws)
    assert rde.device_status(cfg, ws) == 0
    tok = torch.cat((rt.long(), torch.arange(T * shared, device="cuda")))
    q, s = rde.quantize_fp4(x, fmt, g)
    rq, rs = plain.quantize(x, fmt, 1.0 if g is None else float(g))
    assert torch.equal(q, rq) and torch.equal(s, rs)
    assert torch.equal(xq, q[tok]) and torch.equal(xs, s[tok])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,h,I,shared", [(5, 1280, 256, 1), (200, 2304, 768, 0)])
def test_forward_with_wide_rows(fmt, T, h, I, shared):
    """As the layer's test at h = 256: within 2e-2 of fp64 as a whole, each row within twice that."""
    E, k = 8, 2
    ex = Experts(E, h, I, fmt, shared, seed=h, sigma=0.02)
    cfg = ex.config(T, k, renorm=True)
    x = torch.randn(T, h, generator=rng(8), device="cuda").to(torch.bfloat16)
    layer = rde.MoeLayer(cfg, ex.weights, fp4_activations=ex.act or rde.Fp4Activations())
    y = layer(x)
    assert rde.device_status(cfg, layer.ws) == 0
    idx = rde.ws_view(layer.ws, cfg, "topk_idx", torch.int32, (T, k))
    w = rde.ws_view(layer.ws, cfg, "topk_w", torch.float32, (T, k))
    ref = layer_reference(ex, x, idx, w)
    assert (y.double() - ref).norm() <= 2e-2 * ref.norm()
    assert ((y.double() - ref).abs().amax(1) / ref.abs().amax(1)).amax() <= 4e-2


@pytest.mark.parametrize("fmt", FORMATS)
def test_expert_ffn_of_real_size(fmt):
    """h 7168, I 2048, from no row to more than a tile an expert: H code by code against fp64, yd from the H that was
    written, and the same bits again over a workspace of anything."""
    h, I, counts = 7168, 2048, [0, 1, 40, 128, 135]
    E, R = len(counts), sum(counts)
    ex = Experts(E, h, I, fmt, 0, seed=1, sigma=0.02)
    cfg = ex.config(R, 1)
    x = torch.randn(R, h, generator=rng(3), device="cuda")
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    weight = torch.rand(R, generator=rng(6), device="cuda")
    q, s, ws, yd = run_ffn(ex, cfg, x, offsets, weight)
    hq, hs = (v.clone() for v in hidden_of(ws, cfg, R, I, fmt))
    for _ in range(3):
        ws.fill_(255)
        rde.device_status(cfg, ws)
        again = torch.full_like(yd, float("nan"))
        rde.expert_ffn_fp4(cfg, ex.weights, ex.act, q, s, offsets, weight, again, ws)
        assert torch.equal(again, yd)
    xv = plain.values(q, s, fmt, ex.g_x)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        hv = check_hidden(hq[a:b], hs[a:b], xv[a:b], ex.gu[e], I, fmt, ex.g_h)
        w = weight[a:b].double().unsqueeze(1)
        ref, mag = hv @ ex.d[e].T * w, hv.abs() @ ex.d[e].abs().T * w
        tol = product_tolerance(ref, mag, I, torch.bfloat16) + 2.0 ** -23 * ref.abs()
        assert (yd[a:b].double() - ref).abs().sub(tol).amax() <= 0, (e, b - a)
