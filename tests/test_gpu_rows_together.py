"""The operators around the experts used together, as a training step and as an 8-bit layer use them, and the ways in which
calls meet: streams, graphs, threads, buffers that are written in place."""
import importlib.util
import os
import threading

import pytest
import torch

import plain_rows as plain
import routing_dispatch_expert_gb300 as rde
from plain_rows import HALF, U32
from routing_dispatch_expert_gb300 import build as pkg_build
from routing_dispatch_expert_gb300 import moe

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def load_example():
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(EXAMPLES, "train_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_runs():
    history, layer = load_example().main(steps=3, T=300, h=256, E=8, k=2, I=128)
    assert all(l == l and b > 0 for l, b in history)
    assert all(torch.isfinite(p.grad).all() and p.grad.abs().sum() > 0 for p in layer.parameters())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("factor", [0.0, 1.0])
def test_a_training_steps_gradients(score, factor):
    """The whole step in fp32 against the same step in 64 bits by autograd of plain torch operations. Both are sums of smooth
    functions of inputs of size 1 through products of length 256 and less: the fp32 side is off by about 256 u of the largest
    gradient a layer, five layers deep (2^-13.7); 2^-13 of each gradient's largest number is allowed. The selection is the library's."""
    torch.manual_seed(1)
    T, h, E, k, I = 200, 256, 8, 3, 128
    layer = load_example().Layer(h, E, k, I, score, factor).cuda()
    x = torch.randn(T, h, device="cuda", requires_grad=True)
    dy = torch.randn(T, h, device="cuda")
    out, balance = layer(x, alpha=0.1)
    ((out * dy).sum() + balance).backward()

    cfg = rde.make_config(T=T, **layer.shape)
    p = {n: v.detach().double().requires_grad_() for n, v in layer.named_parameters()}
    xd = x.detach().double().requires_grad_()
    y = xd * torch.rsqrt(xd.pow(2).mean(1, keepdim=True) + 1e-6) * p["norm"]
    z = y @ p["router"].T
    idx, _ = rde.route_weights(cfg, (rde.rms_norm(x.detach(), layer.norm.detach()) @ layer.router.detach().T))
    inv = rde.sort_tokens(cfg, idx)["inv_pos"]
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    w = s.gather(1, idx.long())
    w = w / w.sum(1, keepdim=True)
    prob = s / s.sum(1, keepdim=True)
    counts = torch.zeros(E, device="cuda", dtype=torch.float64).index_add_(0, idx.flatten().long(), torch.ones(T * k, device="cuda").double())
    want_balance = 0.1 * E / (k * T) * (counts * prob.mean(0)).sum()
    want = xd.clone()
    for j in range(k):
        gate, up = torch.einsum("th,tih->ti", y, p["gate_up"][idx[:, j].long()]).chunk(2, -1)
        o = torch.einsum("ti,thi->th", torch.nn.functional.silu(gate) * up, p["down"][idx[:, j].long()])
        want = want + torch.where((inv[:, j] >= 0).unsqueeze(1), w[:, j:j + 1] * o, 0.0)
    ((want * dy.double()).sum() + want_balance).backward()
    assert (out.double() - want).abs().max() <= 2 ** -13 * want.abs().max()
    assert abs(float(balance.detach()) - float(want_balance.detach())) <= 2 ** -13 * float(want_balance.detach())
    for name, v in list(layer.named_parameters()) + [("x", x)]:
        ref = xd.grad if name == "x" else p[name].grad
        assert (v.grad.double() - ref).abs().max() <= 2 ** -13 * ref.abs().max(), name


def test_an_8_bit_layers_step():
    """Norm to 8 bits -> route -> sort -> 8-bit rows -> FP8 experts -> back onto the stream. Each expert row against the SwiGLU FFN
    in 64 bits of the values that its codes and its expert's stand for: the product inside is quantised to e4m3, each of
    its numbers off by at most 2^-4 of itself (and 2^-10 of its block's scale, amax / 448: below 2^-18 of the row's largest),
    fp32 sums and bf16 rounding add 2^-8; so 1.1 * 2^-4 of the sum of magnitudes is allowed."""
    torch.manual_seed(2)
    T, h, E, k, I = 333, 512, 16, 4, 256
    cfg = rde.make_config(T=T, h=h, E=E, k=k, I=I, dtype="fp8", score="softmax", renorm=True)
    x, r = (torch.randn(T, h, device="cuda").to(BF16) for _ in range(2))
    w_gu, s_gu = rde.quantize_weights_fp8((torch.randn(E, 2 * I, h, device="cuda") * 0.05).to(BF16))
    w_d, s_d = rde.quantize_weights_fp8((torch.randn(E, h, I, device="cuda") * 0.05).to(BF16))
    weights = rde.Weights(w_router=torch.randn(E, h, device="cuda") * 0.05, w_gu=w_gu, s_gu=s_gu, w_d=w_d, s_d=s_d)
    ws = rde.alloc_workspace(cfg)
    rde.device_status(cfg, ws)
    n = rde.rms_norm_fp8(x, 1 + 0.1 * torch.randn(h, device="cuda"), r, with_y=True)
    idx, tw = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    rde.route(cfg, n["y"], weights, idx, tw, ws=ws)
    s = rde.sort_tokens(cfg, idx)
    xd, xs = rde.permute(cfg, n["q"], s["inv_pos"], s["offsets"], scales=n["s"])
    yd = torch.empty(T * k, h, dtype=BF16, device="cuda")
    rde.expert_ffn(cfg, weights, xd, xs, s["offsets"], torch.ones(T * k, device="cuda"), yd, ws)
    got = rde.unpermute(cfg, yd, s["inv_pos"], tw, base=n["total"])
    assert rde.device_status(cfg, ws) == 0

    value = lambda q, s, n: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(n, -2).repeat_interleave(128, -1)  # noqa: E731
    rows, gu, down = value(xd, xs, 1), value(w_gu, s_gu, 128), value(w_d, s_d, 128)
    assert torch.equal(rows, value(n["q"], n["s"], 1)[s["row_token"].long()])
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), s["counts"].long())
    gate, up = torch.einsum("rh,rih->ri", rows, gu[expert]).chunk(2, -1)
    H = torch.nn.functional.silu(gate) * up
    want, size = (torch.einsum("ri,rhi->rh", a, b) for a, b in ((H, down[expert]), (H.abs(), down[expert].abs())))
    assert ((yd.double() - want).abs() <= 1.1 * 2.0 ** -4 * size).all()
    y, size = plain.unpermute(yd, s["inv_pos"], tw, n["total"])
    assert ((got.double() - y).abs() <= (k + 2) * U32 * size + HALF[BF16] * y.abs() * (1 + 2.0 ** -8)).all()


def run_all(cfg, x, r, w, idx, tw, z, dy):
    """One of each call; everything it returns."""
    y, total = rde.rms_norm(x, w, r)
    q = rde.rms_norm_fp8(x, w, r)
    g = rde.rms_norm_backward(dy, total, w, dtotal=r)
    s = rde.sort_tokens(cfg, idx, tw)
    xd = rde.permute(cfg, y, s["inv_pos"], s["offsets"])
    xq, xs = rde.permute(cfg, q["q"], s["inv_pos"], s["offsets"], q["s"])
    back = rde.unpermute(cfg, xd, s["inv_pos"], tw, base=total)
    dyd, dw = rde.unpermute_backward(cfg, dy, xd, s["inv_pos"], s["offsets"], tw)
    return [y, total, q["q"], q["s"], *g, *s.values(), xd, xq, xs, back, dyd, dw, rde.route_backward(cfg, z, idx, dw)]


def inputs(seed, T=900, cols=1000, E=32, k=4):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    cfg = rde.make_config(T=T, h=256, E=E, k=k, I=256, score="sigmoid", renorm=True, capacity_factor=1.2)
    z = n(T, E)
    idx = torch.topk(z, k).indices.int()
    idx[::7] = -1
    return [cfg, n(T, cols).to(BF16), n(T, cols).to(BF16), n(cols).to(BF16), idx, torch.rand(T, k, generator=gen, device="cuda"), z,
            n(T, cols).to(BF16)]


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_streams_and_threads():
    """Calls on streams of their own, at once and from several host threads: the bits of calls one after the other."""
    sets = [inputs(s) for s in range(4)]
    want = [run_all(*a) for a in sets]
    torch.cuda.synchronize()
    got = [[None] * 5 for _ in sets]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for n in range(5):
                got[i][n] = run_all(*sets[i])
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same(g, want[i]) for i in range(4) for g in got[i])


def test_graphs():
    """Two captured graphs of the same calls, replayed in turn with new inputs."""
    a, b = inputs(10), inputs(11)
    want = [run_all(*v) for v in (a, b)]
    static = [v.clone() if isinstance(v, torch.Tensor) else v for v in a]
    run_all(*static)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], [None, None]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            outs[i] = run_all(*static)
    for i, source in enumerate((b, a, b)):
        for u, v in zip(static[1:], source[1:]):
            u.copy_(v)
        graphs[i % 2].replay()
        assert same(outs[i % 2], want[0 if source is a else 1])


def test_captured_training_step():
    """Forward and backward of the differentiable calls captured into one graph, on leaves of their own."""
    cfg, x, r, w, idx, tw, z, dy = inputs(12)
    static = [v.clone().requires_grad_() for v in (x, r, w, tw, z)]

    def step():
        x, r, w, tw, z = static
        chosen, weights = rde.route_weights(cfg, z)
        y, total = rde.rms_norm(x, w, r)
        s = rde.sort_tokens(cfg, idx)
        xd = rde.permute(cfg, y, s["inv_pos"], s["offsets"])
        out = rde.unpermute(cfg, xd, s["inv_pos"], tw * weights, total, s["offsets"])
        return torch.autograd.grad((out.float() * dy.float()).sum(), static)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for v in got:
        v.zero_()
    graph.replay()
    assert same(got, want)


@pytest.mark.parametrize("cols", [64, 1000, 1003, 4101])
def test_in_place(cols):
    """Through the C entry points: total written over the residual, y over x; dx over dy; y of unpermute over its base."""
    cfg, x, r, w, idx, tw, z, dy = inputs(13, cols=cols)
    lib, n, c = rde.load(), x.shape[0], x.shape[1]
    y, total = rde.rms_norm(x, w, r)
    dx, _, dw = rde.rms_norm_backward(dy, total, w, dtotal=r)
    p = lambda t: t.data_ptr()  # noqa: E731
    x2, r2 = x.clone(), r.clone()
    assert lib.moe_rms_norm(p(x2), 1, n, c, c, p(r2), 1, c, p(w), 1, 1e-6, p(x2), p(r2), None, None, moe._stream()) == 0
    assert torch.equal(x2, y) and torch.equal(r2, total)
    ws = rde.rms_norm_backward_workspace(n, c)
    for over in (0, 1, 2):
        a = [dy.clone(), total.clone(), r.clone()]
        dw2 = torch.empty_like(w)
        assert lib.moe_rms_norm_backward(p(a[0]), 1, n, c, p(a[1]), 1, c, p(a[2]), p(w), 1, 1e-6, p(a[over]), None, p(dw2), p(ws),
                                         ws.numel(), moe._stream()) == 0
        assert torch.equal(a[over], dx) and torch.equal(dw2, dw)
    s = rde.sort_tokens(cfg, idx)
    xd = rde.permute(cfg, y, s["inv_pos"], s["offsets"])
    want = rde.unpermute(cfg, xd, s["inv_pos"], tw, base=total)
    import ctypes
    assert lib.moe_unpermute(ctypes.byref(cfg), p(xd), 1, c, p(s["inv_pos"]), p(tw), p(total), p(total), moe._stream()) == 0
    assert torch.equal(total, want)


def test_launches():
    """The launches that the header says."""
    cfg, x, r, w, idx, tw, z, dy = inputs(14)
    calls = []

    def count(f, n):
        before = rde.launch_count()
        out = f()
        calls.append((rde.launch_count() - before, n))
        return out

    y, total = count(lambda: rde.rms_norm(x, w, r), 1)
    count(lambda: rde.rms_norm_fp8(x, w, r), 1)
    count(lambda: rde.rms_norm_backward(dy, total, w), 2)
    count(lambda: rde.rms_norm_backward(dy, total, None), 1)
    s = count(lambda: rde.sort_tokens(cfg, idx, tw), 2)
    small = rde.make_config(T=512, h=256, E=32, k=4, I=256)
    count(lambda: rde.sort_tokens(small, idx[:512].contiguous()), 1)
    xd = count(lambda: rde.permute(cfg, y, s["inv_pos"], s["offsets"]), 1)
    count(lambda: rde.unpermute(cfg, xd, s["inv_pos"], tw), 1)
    count(lambda: rde.unpermute_backward(cfg, dy, xd, s["inv_pos"], s["offsets"], tw), 1)
    count(lambda: rde.route_backward(cfg, z, idx, tw), 1)
    assert all(a == b for a, b in calls), calls


def test_nothing_outside_the_outputs_is_written():
    """Outputs in the middle of larger buffers: what lies around them stays."""
    T, E, k = 70, 8, 2
    cfg = rde.make_config(T=T, h=256, E=E, k=k, I=256)
    idx = torch.topk(torch.randn(T, E, device="cuda"), k).indices.int()
    s = rde.sort_tokens(cfg, idx)
    lib, st = rde.load(), moe._stream()
    import ctypes
    for cols in (8, 33, 256, 1003, 4104):
        for kind in (F32, BF16):
            t = 0 if kind is F32 else 1

            def framed(n, m):
                pad = 16
                full = torch.full((n * m + 2 * pad,), 7.0, device="cuda", dtype=kind)
                return full, full[pad:pad + n * m].view(n, m), lambda: bool((full[:pad] == 7).all() and (full[pad + n * m:] == 7).all())

            x = torch.randn(T, cols, device="cuda").to(kind)
            w = torch.ones(cols, device="cuda", dtype=kind)
            _, y, ok_y = framed(T, cols)
            _, total, ok_t = framed(T, cols)
            assert lib.moe_rms_norm(x.data_ptr(), t, T, cols, cols, x.data_ptr(), t, cols, w.data_ptr(), t, 1e-6, y.data_ptr(),
                                    total.data_ptr(), None, None, st) == 0
            _, dx, ok_dx = framed(T, cols)
            _, dw, ok_dw = framed(1, cols)
            ws = rde.rms_norm_backward_workspace(T, cols)
            assert lib.moe_rms_norm_backward(x.data_ptr(), t, T, cols, total.data_ptr(), t, cols, None, w.data_ptr(), t, 1e-6,
                                             dx.data_ptr(), None, dw.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
            _, xd, ok_xd = framed(T * k, cols)
            assert lib.moe_permute(ctypes.byref(cfg), x.data_ptr(), kind.itemsize, cols, cols, None, s["inv_pos"].data_ptr(),
                                   s["offsets"].data_ptr(), xd.data_ptr(), None, st) == 0
            _, back, ok_b = framed(T, cols)
            assert lib.moe_unpermute(ctypes.byref(cfg), xd.data_ptr(), t, cols, s["inv_pos"].data_ptr(), None, None,
                                     back.data_ptr(), st) == 0
            _, dyd, ok_d = framed(T * k, cols)
            assert lib.moe_unpermute_backward(ctypes.byref(cfg), x.data_ptr(), None, t, cols, s["inv_pos"].data_ptr(),
                                              s["offsets"].data_ptr(), None, dyd.data_ptr(), None, st) == 0
            assert ok_y() and ok_t() and ok_dx() and ok_dw() and ok_xd() and ok_b() and ok_d(), (cols, kind)
            y2, t2 = rde.rms_norm(x, w, x)
            assert torch.equal(y, y2) and torch.equal(total, t2)
            assert torch.equal(xd, rde.permute(cfg, x, s["inv_pos"], s["offsets"]))
            assert torch.equal(back, rde.unpermute(cfg, xd, s["inv_pos"]))


def test_numbers_of_the_other_rows_do_not_show():
    """A row's norm and gradient do not depend on the rows beside it, whatever they hold (odd rows are read with the bytes
    around them)."""
    for cols in (33, 1003, 4101):
        for kind in (F32, BF16):
            x = torch.randn(40, cols, device="cuda").to(kind)
            dy = torch.randn(40, cols, device="cuda").to(kind)
            want = rde.rms_norm_backward(dy, x, None)[0]
            bad, dbad = x.clone(), dy.clone()
            bad[1::2], dbad[1::2] = float("nan"), float("inf")
            got = rde.rms_norm_backward(dbad, bad, None)[0]
            assert torch.equal(got[::2], want[::2]) and got[1::2].isnan().all()
            assert torch.equal(rde.rms_norm(bad)[::2], rde.rms_norm(x)[::2])
