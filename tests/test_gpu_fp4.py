"""Microscaled 4-bit rows, products and experts on the GPU against their definitions in 64 bits (plain_fp4)."""
import numpy as np
import pytest
import torch

import plain_fp4 as plain
import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build

pytestmark = pytest.mark.gpu

FORMATS = ("nvfp4", "mxfp4")
TYPES = (torch.float32, torch.bfloat16, torch.float16)


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def scale_of(x, fmt):
    """(tensor or None, number): a matrix scale as a user would choose it."""
    if fmt == "mxfp4":
        return None, 1.0
    g = (x.float().abs().amax() / 2688).clamp(min=1e-30).reshape(1)
    return g, float(g)


# ------------------------------------------------------------------------------------------
# quantise, and back: codes, scales and values are equal to the definition's, bit for bit
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (257, 2080), (64, 7168)])
def test_quantize_and_back(fmt, dtype, rows, cols):
    x = torch.randn(rows, cols, generator=rng(rows + cols), device="cuda")
    x = (x * torch.exp(2 * torch.randn(1, cols, generator=rng(5), device="cuda"))).clamp(-6e4, 6e4).to(dtype)
    x[0, :16] = 0
    x[-1, 5] = -0.0
    gt, g = scale_of(x, fmt)
    q, s = rde.quantize_fp4(x, fmt, gt)
    rq, rs = plain.quantize(x, fmt, g)
    assert torch.equal(s, rs) and torch.equal(q, rq)
    want = plain.values(rq, rs, fmt, g)
    for out in TYPES:
        # values have at most 7 bits times g: rounded to fp32, then to the output's type
        assert torch.equal(rde.dequantize_fp4(q, s, fmt, gt, dtype=out), want.float().to(out)), out


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_tie_goes_to_the_even_code(fmt):
    """Values halfway between two codes, and one fp32 step to either side, with a power-of-two step."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    inf = torch.full_like(mids, float("inf"))
    v = torch.cat((mids, torch.nextafter(mids, inf), torch.nextafter(mids, -inf), mids.new_tensor([6.0, 7.9, 0.0])))
    block = torch.zeros(4, plain.BLOCK[fmt], device="cuda")
    block[:, 0] = 6.0 if fmt == "nvfp4" else 4.0  # the scale is 1
    block[:, 1:13] = torch.cat((v, -v)).view(4, -1)
    x = block.view(1, -1) if fmt == "mxfp4" else block.view(2, 32)
    q, s = rde.quantize_fp4(x, fmt)
    rq, rs = plain.quantize(x, fmt)
    assert torch.equal(q, rq) and torch.equal(s, rs)


@pytest.mark.parametrize("fmt", FORMATS)
def test_extreme_blocks(fmt):
    """Zeros, the smallest and largest numbers, infinities and NaN: a block that is not finite is NaN, the
    others of its row are not touched by it."""
    n = plain.BLOCK[fmt]
    x = torch.randn(8, 4 * n, generator=rng(9), device="cuda")
    x[0] = 0
    x[1] = 1e-45
    x[2] = 3e38
    x[3, n + 3] = float("inf")
    x[4, 2 * n + 1] = float("nan")
    x[5, 0] = -float("inf")
    x[6] = 2.0 ** -126
    q, s = rde.quantize_fp4(x, fmt)
    rq, rs = plain.quantize(x, fmt)
    assert torch.equal(s, rs) and torch.equal(q, rq)
    v = rde.dequantize_fp4(q, s, fmt)
    bad = torch.isnan(v).view(8, 4, n)
    for r, b in ((3, 1), (4, 2), (5, 0)):
        assert bad[r, b].all() and int(bad[r].sum()) == n
    assert int(bad.sum()) == 3 * n


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_rows(fmt):
    big = torch.randn(33, 256 + 64, generator=rng(4), device="cuda").to(torch.bfloat16)
    x = big[::3, 8:8 + 256]
    q, s = rde.quantize_fp4(x, fmt)
    rq, rs = rde.quantize_fp4(x.contiguous(), fmt)
    assert torch.equal(q, rq) and torch.equal(s, rs)
    with pytest.raises(rde.MoeError):
        rde.quantize_fp4(big[:, 1:257], fmt)  # 2 bytes off: not 16-byte aligned
    with pytest.raises(ValueError):
        rde.quantize_fp4(big.T, fmt)


def test_empty_rows():
    q, s = rde.quantize_fp4(torch.empty(0, 64, device="cuda"), "mxfp4")
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert rde.dequantize_fp4(q, s, "mxfp4").shape == (0, 64)


def test_weights_quantiser_agrees():
    """NVFP4 rows with the weights' own matrix scale are what moe_quantize_weights_nvfp4 makes of them."""
    w = (torch.randn(96, 512, generator=rng(2), device="cuda") * 0.02).to(torch.bfloat16)
    q, s, g = rde.quantize_weights_nvfp4(w)
    q2, s2 = rde.quantize_fp4(w, "nvfp4", g)
    assert torch.equal(q, q2) and torch.equal(s, s2)


# ------------------------------------------------------------------------------------------
# the product
# ------------------------------------------------------------------------------------------
def operand(rows, cols, fmt, seed, sigma=1.0):
    x = torch.randn(rows, cols, generator=rng(seed), device="cuda") * sigma
    gt, g = scale_of(x, fmt)
    q, s = rde.quantize_fp4(x, fmt, gt)
    return q, s, gt, plain.values(q, s, fmt, g)


def product_tolerance(ref, abs_sum, K, dtype):
    """Sums of exact products: K additions, each off by at most 2^-23 of the sum of magnitudes (truncation, in any
    order); the two matrix scales and the factor round three times; then half a step of the output."""
    u = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    return K * 2.0 ** -23 * abs_sum + (u + 4 * 2.0 ** -24) * ref.abs() + 1e-30


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 256, 256), (2, 17, 64), (31, 255, 96), (33, 257, 320), (64, 7168, 2048),
                                   (97, 128, 288), (128, 256, 512), (129, 600, 2080), (300, 513, 4096), (1, 7168, 2048),
                                   (1000, 1030, 1056)])
def test_matmul(fmt, M, N, K):
    aq, a_s, ga, a = operand(M, K, fmt, 1)
    bq, b_s, gb, b = operand(N, K, fmt, 2, 0.02)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        rde.matmul_fp4(aq, a_s, bq, b_s, fmt, ga, gb, y=y, status=status)
        assert (y.double() - ref).abs().sub(product_tolerance(ref, mag, K, dtype)).amax() <= 0
    assert int(status) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_matmul_scales_reach_their_rows(fmt):
    """Every row of A and B, and every block along K, has a scale of its own (powers of two over a wide range): a
    scale that is read from another row or block is off by a factor of two at least."""
    M, N, K = 140, 300, 768
    n = plain.BLOCK[fmt]
    gen = rng(11)

    def one(rows):
        x = torch.sign(torch.randn(rows, K, generator=gen, device="cuda")) * 4
        e = torch.randint(-3, 4, (rows, K // n), generator=gen, device="cuda")
        return rde.quantize_fp4(x * torch.exp2(e.float()).repeat_interleave(n, 1), fmt)

    (aq, a_s), (bq, b_s) = one(M), one(N)
    a, b = plain.values(aq, a_s, fmt), plain.values(bq, b_s, fmt)
    y = rde.matmul_fp4(aq, a_s, bq, b_s, fmt, dtype=torch.float32)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    assert (y.double() - ref).abs().sub(product_tolerance(ref, mag, K, torch.float32)).amax() <= 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 10001, 96), (33, 9985, 544), (130, 5130, 800), (640, 2304, 2080)])
def test_matmul_with_more_tiles_than_run_narrow(fmt, M, N, K):
    """Products whose 64-column tiles would not all run at once: 256-column tiles, with one and several row tiles."""
    aq, a_s, ga, a = operand(M, K, fmt, 1)
    bq, b_s, gb, b = operand(N, K, fmt, 2, 0.02)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    for dtype in (torch.bfloat16, torch.float32):
        y = rde.matmul_fp4(aq, a_s, bq, b_s, fmt, ga, gb, dtype=dtype)
        assert (y.double() - ref).abs().sub(product_tolerance(ref, mag, K, dtype)).amax() <= 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(140, 300, 4608), (140, 5000, 4608), (256, 4864, 1024)])
def test_matmul_scales_of_long_rows(fmt, M, N, K):
    """As above in narrow and wide tiles, with several fills of the scales' ring: a scale of another row, block or fill
    is off by a factor of two at least."""
    n = plain.BLOCK[fmt]
    gen = rng(12)

    def one(rows):
        x = torch.sign(torch.randn(rows, K, generator=gen, device="cuda")) * 4
        e = torch.randint(-3, 4, (rows, K // n), generator=gen, device="cuda")
        return rde.quantize_fp4(x * torch.exp2(e.float()).repeat_interleave(n, 1), fmt)

    (aq, a_s), (bq, b_s) = one(M), one(N)
    a, b = plain.values(aq, a_s, fmt), plain.values(bq, b_s, fmt)
    y = rde.matmul_fp4(aq, a_s, bq, b_s, fmt, dtype=torch.float32)
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    assert (y.double() - ref).abs().sub(product_tolerance(ref, mag, K, torch.float32)).amax() <= 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_matmul_writes_nothing_else(fmt):
    """Rows of an output with gaps: the gaps, and the rows before and after, keep what they held."""
    M, N, K = 130, 70, 160
    aq, a_s, ga, a = operand(M, K, fmt, 1)
    bq, b_s, gb, b = operand(N, K, fmt, 2)
    big = torch.full((M + 2, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    rde.matmul_fp4(aq, a_s, bq, b_s, fmt, ga, gb, y=big[1:-1, 16:16 + N])
    assert (big[0] == 7).all() and (big[-1] == 7).all() and (big[:, :16] == 7).all() and (big[:, 16 + N:] == 7).all()
    ref = a @ b.T
    tol = product_tolerance(ref, a.abs() @ b.abs().T, K, torch.bfloat16)
    assert (big[1:-1, 16:16 + N].double() - ref).abs().sub(tol).amax() <= 0


def test_matmul_carries_nan_of_its_rows_only():
    fmt, M, N, K = "mxfp4", 40, 50, 256
    x = torch.randn(M, K, generator=rng(1), device="cuda")
    x[7, 100] = float("inf")
    aq, a_s = rde.quantize_fp4(x, fmt)
    bq, b_s, _, _ = operand(N, K, fmt, 2)
    y = rde.matmul_fp4(aq, a_s, bq, b_s, fmt)
    bad = torch.isnan(y)
    assert bad[7].all() and int(bad.sum()) == N


def test_matmul_refuses_other_shapes():
    aq, a_s, _, _ = operand(4, 64, "mxfp4", 1)
    bq, b_s, _, _ = operand(4, 96, "mxfp4", 1)
    with pytest.raises(ValueError, match="rows of 64"):
        rde.matmul_fp4(aq, a_s, bq, b_s, "mxfp4")
    with pytest.raises(ValueError, match="scales must have shape"):
        rde.matmul_fp4(aq, a_s, aq, a_s, "nvfp4")
    with pytest.raises(ValueError, match="ga must have shape"):
        rde.matmul_fp4(aq, a_s, aq, a_s, "mxfp4", ga=torch.ones(2, device="cuda"))


# ------------------------------------------------------------------------------------------
# the experts
# ------------------------------------------------------------------------------------------
class Experts:
    """Quantised weights of a layer and their fp64 values."""

    def __init__(self, E, h, I, fmt, shared, seed=0, sigma=0.05):
        self.E, self.h, self.I, self.fmt, self.shared = E, h, I, fmt, shared
        gen = rng(seed + 1)
        t, self.gu, self.d = {}, [], []
        for name, rows, cols, vals in (("gu", 2 * I, h, self.gu), ("d", h, I, self.d)):
            w = (torch.randn(E + shared, rows, cols, generator=gen, device="cuda") * sigma).to(torch.bfloat16)
            if fmt == "nvfp4":
                q, s, g = rde.quantize_weights_nvfp4(w)
            else:
                q, s = (v.view(E + shared, rows, -1) for v in rde.quantize_fp4(w.view(-1, cols), fmt))
                g = torch.ones(E + shared, device="cuda")
            vals += [plain.values(q[e], s[e], fmt, float(g[e])) for e in range(E + shared)]
            t["w_" + name], t["s_" + name] = q[:E].contiguous(), s[:E].contiguous()
            if shared:
                t[f"w_{name}_shared"], t[f"s_{name}_shared"] = q[E].clone(), s[E].clone()
            if fmt == "nvfp4":
                t["g_" + name] = g[:E].clone()
                if shared:
                    t[f"g_{name}_shared"] = g[E:].clone()
        self.w_router = torch.randn(E, h, generator=gen, device="cuda") * 0.05
        self.weights = rde.Weights(w_router=self.w_router, **t)
        self.act, self.g_x, self.g_h = None, 1.0, 1.0
        if fmt == "nvfp4":
            gx, gh = torch.tensor([[4.5 / 2688], [40.0 / 2688]], device="cuda")
            self.act, self.g_x, self.g_h = rde.Fp4Activations(gx, gh), float(gx), float(gh)

    def config(self, T, k, **kw):
        return rde.make_config(T=T, h=self.h, E=self.E, k=k, I=self.I, I_shared=self.I if self.shared else 0,
                               dtype=self.fmt, **kw)


def hidden_of(ws, cfg, rows, I, fmt):
    """(codes, scales) of H in the workspace."""
    off = rde.workspace_layout(cfg)["hbuf"]
    n, m = rows * I // 2, rows * I // plain.BLOCK[fmt]
    at = off + (n + 255) // 256 * 256
    return ws[off:off + n].view(rows, I // 2), ws[at:at + m].view(rows, I // plain.BLOCK[fmt])


def check_hidden(hq, hs, x, gu, I, fmt, g):
    """H codes and scales of some rows against fp64: each value is the nearest of its block's grid, up to the error of
    the fp32 product: K additions of 2^-23 of the magnitudes in gate and up, and SiLU from exp and a quotient, at most
    (6 + 2 |gate|) 2^-23 relative."""
    K = x.shape[1]
    p, mag = x @ gu.T, x.abs() @ gu.abs().T
    gate, up = p.split(I, 1)
    mg, mu = (mag * (K * 2.0 ** -23)).split(I, 1)
    h = plain.silu(gate) * up
    err = 1.1 * mg * up.abs() + plain.silu(gate).abs() * mu + mg * mu + (8 + 2 * gate.abs()) * 2.0 ** -23 * h.abs() + 1e-30
    n = plain.BLOCK[fmt]
    amax = h.abs().view(len(h), -1, n).amax(-1)
    slack = err.view(len(h), -1, n).amax(-1)
    low, high = (torch.clamp(amax - slack, min=0), amax + slack)
    if fmt == "nvfp4":
        codes = [plain.nearest(plain.E4M3, v / (6 * g) * f) for v, f in ((low, 1 - 2.0 ** -22), (high, 1 + 2.0 ** -22))]
    else:
        codes = [torch.where(v > 0, torch.frexp(v)[1] + 124, 0).clamp(min=0) for v in (low, high)]
    assert ((hs.long() >= codes[0]) & (hs.long() <= codes[1])).all()
    step = (plain.scale_values(hs, fmt) * g).repeat_interleave(n, 1)
    y = torch.where(step > 0, h / torch.where(step > 0, step, 1.0), 0.0)
    got = plain.code_values(hq)
    best = plain.GRID.to(y.device)[plain.nearest(plain.GRID, y.abs())] * torch.sign(y)
    worse = (got - y).abs() - (best - y).abs()
    room = torch.where(step > 0, 2 * err / torch.where(step > 0, step, 1.0), 0.0) + 2.0 ** -22 * y.abs()
    assert (worse <= room).all()
    return plain.values(hq, hs, fmt, g)


def run_ffn(ex, cfg, x, offsets, row_weight):
    """yd and the workspace of moe_expert_ffn_fp4 on rows x (fp32)."""
    q, s = rde.quantize_fp4(x, ex.fmt, None if ex.act is None else ex.act.tensors[0])
    ws = rde.alloc_workspace(cfg)
    rde.device_status(cfg, ws)
    yd = torch.full((x.shape[0], ex.h), float("nan"), dtype=torch.bfloat16, device="cuda")
    rde.expert_ffn_fp4(cfg, ex.weights, ex.act, q, s, offsets, row_weight, yd, ws)
    assert rde.device_status(cfg, ws) == 0
    return q, s, ws, yd


COUNTS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 0, 255, 256, 257, 300]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("h,I,shared", [(256, 256, 0), (512, 256, 1), (768, 512, 0)])
def test_expert_ffn_at_every_tile_edge(fmt, h, I, shared):
    E, R = len(COUNTS), sum(COUNTS)
    ex = Experts(E, h, I, fmt, shared, seed=h)
    T = R  # k = 1: one row a token
    cfg = ex.config(T, 1)
    rows = R + (T if shared else 0)
    x = torch.randn(rows, h, generator=rng(3), device="cuda")
    offsets = torch.tensor(np.concatenate(([0], np.cumsum(COUNTS))), dtype=torch.int32, device="cuda")
    weight = torch.rand(rows, generator=rng(6), device="cuda")
    q, s, ws, yd = run_ffn(ex, cfg, x, offsets, weight)
    hq, hs = hidden_of(ws, cfg, rows, I, fmt)
    xv = plain.values(q, s, fmt, ex.g_x)
    groups = [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(E)] + ([(E, R, R + T)] if shared else [])
    for e, a, b in groups:
        if a == b:
            continue
        hv = check_hidden(hq[a:b], hs[a:b], xv[a:b], ex.gu[e], I, fmt, ex.g_h)
        w = weight[a:b].double().unsqueeze(1) if e < E else 1.0
        ref, mag = hv @ ex.d[e].T * w, hv.abs() @ ex.d[e].abs().T * w
        tol = product_tolerance(ref, mag, I, torch.bfloat16) + 2.0 ** -23 * ref.abs()
        assert (yd[a:b].double() - ref).abs().sub(tol).amax() <= 0, (e, b - a)


def layer_reference(ex, x, idx, w):
    """The layer in fp64 with 4-bit rows, from the router's choices."""
    T, k = idx.shape
    gx = ex.g_x
    xv = plain.values(*plain.quantize(x, ex.fmt, gx), ex.fmt, gx)

    def ffn(e, rows):
        gate, up = (rows @ ex.gu[e].T).split(ex.I, 1)
        h = plain.silu(gate) * up
        return plain.values(*plain.quantize(h, ex.fmt, ex.g_h), ex.fmt, ex.g_h) @ ex.d[e].T

    y = torch.zeros(T, ex.h, dtype=torch.float64, device=x.device)
    for e in range(ex.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            y.index_add_(0, t, ffn(e, xv[t]) * w[t, j].double().unsqueeze(1))
    return y + ffn(ex.E, xv) if ex.shared else y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k,shared,score", [(1, 8, 2, 1, "softmax"), (5, 8, 1, 0, "sigmoid"), (333, 16, 4, 1, "sigmoid"),
                                                (2000, 130, 3, 0, "softmax"), (700, 160, 8, 1, "sigmoid")])
def test_forward(fmt, T, E, k, shared, score):
    """The layer against fp64; rounding yd and y is 2 x 2^-8 of each row's largest terms, and where fp32 and fp64 round
    H to neighbouring codes an output moves by a step of one of I elements: within the layer's 2e-2 as for bf16."""
    ex = Experts(E, 256, 512, fmt, shared)
    cfg = ex.config(T, k, score=score, renorm=True)
    x = torch.randn(T, 256, generator=rng(8), device="cuda").to(torch.bfloat16)
    layer = rde.MoeLayer(cfg, ex.weights, fp4_activations=ex.act or rde.Fp4Activations())
    y = layer(x)
    assert rde.device_status(cfg, layer.ws) == 0
    idx = rde.ws_view(layer.ws, cfg, "topk_idx", torch.int32, (T, k))
    w = rde.ws_view(layer.ws, cfg, "topk_w", torch.float32, (T, k))
    ref = layer_reference(ex, x, idx, w)
    assert (y.double() - ref).norm() <= 2e-2 * ref.norm()
    err = (y.double() - ref).abs().amax(1) / ref.abs().amax(1)
    assert err.amax() <= 4e-2 and err.median() <= 2e-2
    # the steps one by one give the same bits, and dispatch the same codes as the quantiser
    R_tot = T * k + (T if shared else 0)
    b = plain.BLOCK[fmt]
    i32 = lambda *n: torch.full(n, -5, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, inv, rt = i32(E), i32(E + 1), i32(T, k), i32(T * k)
    rw = torch.empty(T * k, device="cuda")
    xq = torch.zeros(R_tot, 128, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(R_tot, 256 // b, dtype=torch.uint8, device="cuda")
    ws = rde.alloc_workspace(cfg)
    rde.device_status(cfg, ws)
    idx2, w2 = torch.empty_like(idx), torch.empty_like(w)
    rde.route(cfg, x, ex.weights, idx2, w2, ws=ws)
    rde.dispatch_fp4(cfg, ex.act, x, idx2, w2, counts, offsets, inv, rt, rw, xq, xs, ws)
    tok = torch.cat((rt.long(), torch.arange(T, device="cuda"))) if shared else rt.long()
    q, s = rde.quantize_fp4(x, fmt, ex.act.tensors[0] if ex.act else None)
    assert torch.equal(xq, q[tok]) and torch.equal(xs, s[tok])
    yd = torch.empty(R_tot, 256, dtype=torch.bfloat16, device="cuda")
    rde.expert_ffn_fp4(cfg, ex.weights, ex.act, xq, xs, offsets, rw, yd, ws)
    y2 = torch.empty_like(x)
    rde.combine(cfg, yd, inv, y2)
    assert torch.equal(y, y2)


def test_capacity_and_placement():
    """Dropped assignments have no rows, and replicas of an expert give the same outputs as one slot each."""
    fmt, T, E, k = "nvfp4", 600, 16, 4
    ex = Experts(E, 256, 256, fmt, 1)
    x = torch.randn(T, 256, generator=rng(8), device="cuda").to(torch.bfloat16)
    cfg = ex.config(T, k, capacity_factor=0.8)
    layer = rde.MoeLayer(cfg, ex.weights, fp4_activations=ex.act)
    y = layer(x).clone()
    idx = rde.ws_view(layer.ws, cfg, "topk_idx", torch.int32, (T, k))
    w = rde.ws_view(layer.ws, cfg, "topk_w", torch.float32, (T, k))
    inv = rde.ws_view(layer.ws, cfg, "inv_pos", torch.int32, (T, k))
    assert rde.balance(cfg, layer.ws)["dropped"] == int((inv < 0).sum()) > 0
    ref = layer_reference(ex, x, idx, torch.where(inv < 0, 0.0, w))
    assert (y.double() - ref).norm() <= 2e-2 * ref.norm()
    load = torch.bincount(idx.flatten().long(), minlength=E).cpu().numpy()
    placed = ex.config(T, k, capacity_factor=0.8, placement=rde.Placement(rde.eplb_plan(load, 4, 4)))
    assert torch.equal(rde.MoeLayer(placed, ex.weights, fp4_activations=ex.act)(x), y)


def test_no_tokens():
    ex = Experts(8, 256, 256, "mxfp4", 1)
    cfg = ex.config(0, 2)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(rde.workspace_size(cfg), 256), dtype=torch.uint8, device="cuda")
    rde.forward_fp4(cfg, x if x.data_ptr() else ws, ex.weights, None, torch.empty(1, 256, device="cuda"), ws)
    torch.cuda.synchronize()


def test_graph_and_other_streams():
    """Captured into a graph and replayed on new inputs, and run on a stream of its own: the same bits."""
    fmt, T, k = "nvfp4", 150, 2
    ex = Experts(8, 256, 256, fmt, 1)
    cfg = ex.config(T, k)
    xs = [torch.randn(T, 256, generator=rng(i), device="cuda").to(torch.bfloat16) for i in range(3)]
    layer = rde.MoeLayer(cfg, ex.weights, fp4_activations=ex.act)
    want = [layer(x).clone() for x in xs]
    x, y = xs[0].clone(), torch.empty_like(xs[0])
    layer(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, y)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        y.zero_()
        graph.replay()
        assert torch.equal(y, want[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = layer(xs[2])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, want[2])


def test_repeats_bit_for_bit():
    fmt = "nvfp4"
    aq, a_s, ga, _ = operand(333, 1024, fmt, 1)
    bq, b_s, gb, _ = operand(999, 1024, fmt, 2)
    y = rde.matmul_fp4(aq, a_s, bq, b_s, fmt, ga, gb)
    for _ in range(5):
        assert torch.equal(rde.matmul_fp4(aq, a_s, bq, b_s, fmt, ga, gb), y)
