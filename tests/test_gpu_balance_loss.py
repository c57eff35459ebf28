"""The balance loss and its gradient on the GPU against their formulas in 64 bits (plain_fp4)."""
import pytest
import torch

import plain_fp4 as plain
import routing_dispatch_expert_gb300 as rde
from routing_dispatch_expert_gb300 import build as pkg_build

pytestmark = pytest.mark.gpu

ALPHA = 0.01
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg_build.build()
    rde.load()


def config(T, E, k, score):
    return rde.make_config(T=T, h=256, E=E, k=k, I=256, score=score)


def inputs(T, E, k, dtype, seed=0, seqs=1, pad=0.0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(T, E, generator=gen, device="cuda") * spread).to(dtype)
    idx = torch.topk(logits.float(), k).indices.int()
    cuts = torch.randint(0, T + 1, (seqs - 1,), generator=gen, device="cuda").sort().values
    off = torch.cat((cuts.new_zeros(1), cuts, cuts.new_full((1,), T))).int()
    mask = torch.rand(T, generator=gen, device="cuda") >= pad
    return logits, idx, off, mask


def exponent_span(logits):
    """Largest |l - max| (capped: beyond 90 the probability is 0 in fp32 to within 1e-38)."""
    l = logits.double()
    d = (l.amax(-1, keepdim=True) - l)
    return float(d[torch.isfinite(d)].clamp(max=90).amax()) if torch.isfinite(d).any() else 0.0


def probability_error(logits, E):
    """Relative error of one p: two roundings of an exponent of at most x (x 2^-23), ex2.approx (2^-22), the quotient of
    the sigmoid (2^-22 and the sum's 2^-24), in numerator and, averaged, denominator; E additions in the sum; one
    reciprocal and one product. (Sigmoids: exponents of either sign, at most x + max |l| in size.)"""
    l = logits.double()
    top = float(l[torch.isfinite(l)].abs().clamp(max=90).amax()) if torch.isfinite(l).any() else 0.0
    x = exponent_span(logits) + top
    return 2 * (x * 2.0 ** -23 + 3 * 2.0 ** -22) + (E + 4) * U


def check(cfg, logits, idx, off, mask, score, dloss):
    T, E, k = cfg.T, cfg.E, cfg.k
    S = 1 if off is None else len(off) - 1
    out = rde.balance_loss(cfg, logits, idx, ALPHA, off, mask)
    ref = plain.balance_loss(logits, idx, score, ALPHA, off, mask)
    assert torch.equal(out["counts"].long(), ref["counts"].long().cuda())
    assert torch.equal(out["tokens"].cpu().long(), ref["tokens"].long())
    eps = probability_error(logits, E)
    n = ref["tokens"].cuda().double().unsqueeze(1)
    # a mean of n: n additions of positive terms, one quotient
    tol = (eps + (n + 2) * U) * ref["mean_prob"] + 1e-36
    assert ((out["mean_prob"].double() - ref["mean_prob"]).abs() <= tol).all()
    # E products and additions more
    assert ((out["loss"].double() - ref["loss"]).abs() <= (eps + (n[:, 0] + E + 8) * U) * ref["loss"] + 1e-36).all()
    d = rde.balance_loss_backward(cfg, logits, out["counts"], out["tokens"], ALPHA, dloss, off, mask)
    want = plain.balance_loss_backward(logits, ref["counts"].cuda(), k, score, ALPHA, dloss, off, mask)
    # p (c - sum p c): errors of p in both places, the sum's E additions, the factors' roundings; the difference cancels,
    # so they count against the size of its terms, at most the row's largest count
    offs = [0, T] if off is None else [int(v) for v in off]
    bound = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    for s, (a, b) in enumerate(zip(offs[:-1], offs[1:])):
        m = max(int(ref["tokens"][s]), 1)
        p = plain.probabilities(torch.nan_to_num(logits[a:b].float(), nan=0.0), score)
        bound[a:b] = abs(float(dloss[s])) * ALPHA * E / (k * m * m) * p * float(ref["counts"][s].max())
    half = 2.0 ** -8 if logits.dtype == torch.bfloat16 else U
    tol = 3 * (eps + (E + 8) * U) * bound + half * want.abs() + 1e-36
    assert d.dtype == logits.dtype
    assert ((d.double() - want).abs() <= tol).all()
    return out, d


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,seqs,pad", [
    (1, 1, 1, 1, 0.0), (1, 8, 2, 1, 0.0), (7, 3, 2, 3, 0.3), (64, 5, 1, 9, 0.5), (1000, 8, 2, 1, 0.0),
    (3000, 8, 2, 7, 0.1), (333, 16, 4, 2, 0.1), (2049, 30, 3, 5, 0.2), (700, 61, 6, 4, 0.1), (1500, 128, 8, 1, 0.0),
    (1234, 130, 4, 6, 0.1), (5000, 256, 8, 3, 0.1), (511, 257, 8, 40, 0.1), (400, 512, 8, 2, 0.0), (300, 1000, 4, 3, 0.2),
    (200, 1024, 32, 1, 0.0)])
def test_loss_and_gradient(score, dtype, T, E, k, seqs, pad):
    logits, idx, off, mask = inputs(T, E, k, dtype, seed=T + E, seqs=seqs, pad=pad)
    dloss = torch.rand(seqs, device="cuda") * 2 - 0.5
    check(config(T, E, k, score), logits, idx, off, mask, score, dloss)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_batch_without_sequences_or_mask(score):
    T, E, k = 40000, 64, 6
    logits, idx, _, _ = inputs(T, E, k, torch.float32)
    check(config(T, E, k, score), logits, idx, None, None, score, torch.ones(1, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [9, 900])
def test_padding_is_left_out_whatever_it_holds(score, T):
    E, k = 12, 3
    logits, idx, off, mask = inputs(T, E, k, torch.float32, seqs=2, pad=0.4)
    dloss = torch.ones(2, device="cuda")
    cfg = config(T, E, k, score)
    out, d = check(cfg, logits, idx, off, mask, score, dloss)
    dirty = logits.clone()
    dirty[~mask] = float("nan")
    bad_idx = idx.clone()
    bad_idx[~mask] = 1 << 30
    out2 = rde.balance_loss(cfg, dirty, bad_idx, ALPHA, off, mask)
    for name in out:
        assert torch.equal(out[name], out2[name])
    d2 = rde.balance_loss_backward(cfg, dirty, out["counts"], out["tokens"], ALPHA, dloss, off, mask)
    assert torch.equal(d, d2) and (d2[~mask] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [6, 2000])
def test_masked_experts(score, T):
    """-inf masks an expert; a row of nothing but -inf has no probabilities; the lowest number of the type is a
    number: a row of it is even. Very negative rows keep their ratios although every sigmoid underflows."""
    E, k = 8, 2
    logits, idx, _, _ = inputs(T, E, k, torch.float32)
    logits[0, 3:] = -float("inf")
    logits[1] = -float("inf")
    logits[2] = torch.finfo(torch.float32).min
    logits[3] -= 500.0
    logits[4, ::2] = torch.finfo(torch.float32).min
    logits[5] = 80.0
    idx[1] = -1  # no choice: not counted
    out, d = check(config(T, E, k, score), logits, idx, None, None, score, torch.ones(1, device="cuda"))
    assert (d[1] == 0).all() and (d[0, 3:] == 0).all() and torch.isfinite(d).all()
    assert int(out["counts"].sum()) == (T - 1) * k


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_shows(score):
    T, E, k = 50, 8, 2
    logits, idx, _, _ = inputs(T, E, k, torch.float32)
    logits[4, 1] = float("nan")
    cfg = config(T, E, k, score)
    out = rde.balance_loss(cfg, logits, idx, ALPHA)
    assert torch.isnan(out["loss"]).all()
    d = rde.balance_loss_backward(cfg, logits, out["counts"], out["tokens"], ALPHA, torch.ones(1, device="cuda"))
    assert torch.isnan(d[4]).all() and torch.isfinite(d[torch.arange(T, device="cuda") != 4]).all()


def test_empty_sequences_and_no_tokens():
    T, E, k = 100, 8, 2
    logits, idx, _, _ = inputs(T, E, k, torch.float32)
    off = torch.tensor([0, 0, 40, 40, 40, 90, 90], dtype=torch.int32, device="cuda")  # tokens 90 .. are in none
    out, d = check(config(T, E, k, "softmax"), logits, idx, off, None, "softmax", torch.ones(6, device="cuda"))
    assert out["tokens"].tolist() == [0, 40, 0, 0, 50, 0] and (d[90:] == 0).all()
    none = torch.zeros(T, dtype=torch.uint8, device="cuda")
    out = rde.balance_loss(config(T, E, k, "softmax"), logits, idx, ALPHA, off, none)
    assert (out["loss"] == 0).all() and (out["counts"] == 0).all() and (out["mean_prob"] == 0).all()
    cfg = config(0, E, k, "softmax")
    out = rde.balance_loss(cfg, logits[:0], idx[:0], ALPHA, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert float(out["loss"]) == 0 and (out["counts"] == 0).all() and out["tokens"].tolist() == [0]
    assert rde.balance_loss_backward(cfg, logits[:0], out["counts"], out["tokens"], ALPHA,
                                     torch.ones(1, device="cuda")).shape == (0, E)


@pytest.mark.parametrize("T,E,S", [(30000, 8, 3000), (300, 8, 2000), (64, 256, 64), (5000, 64, 900)])
def test_many_sequences_over_many_blocks(T, E, S):
    k = 2
    logits, idx, off, mask = inputs(T, E, k, torch.float32, seqs=S, pad=0.1)
    out = rde.balance_loss(config(T, E, k, "softmax"), logits, idx, ALPHA, off, mask)
    p = plain.probabilities(logits, "softmax")
    seq = torch.bucketize(torch.arange(T, device="cuda"), off[1:].long(), right=True)[mask]
    n = torch.bincount(seq, minlength=S)
    mean = torch.zeros(S, E, dtype=torch.float64, device="cuda").index_add_(0, seq, p[mask]) / n.clamp(min=1).unsqueeze(1)
    assert torch.equal(out["tokens"].long(), n)
    counts = torch.bincount((seq.unsqueeze(1) * E + idx[mask].long()).flatten(), minlength=S * E).view(S, E)
    assert torch.equal(out["counts"].long(), counts)
    assert ((out["mean_prob"].double() - mean).abs() <= (probability_error(logits, E) + (int(n.max()) + 2) * U) * mean + 1e-36).all()


def test_repeats_bit_for_bit_in_a_graph_and_on_other_streams():
    T, E, k = 9000, 64, 6
    logits, idx, off, mask = inputs(T, E, k, torch.float32, seqs=5, pad=0.1)
    cfg = config(T, E, k, "sigmoid")
    ws = rde.balance_loss_workspace(cfg, 5)
    dloss = torch.ones(5, device="cuda")

    def step(z):
        out = rde.balance_loss(cfg, z, idx, ALPHA, off, mask, ws=ws)
        return out, rde.balance_loss_backward(cfg, z, out["counts"], out["tokens"], ALPHA, dloss, off, mask)

    want, dwant = step(logits)
    ws.fill_(255)  # what the workspace holds does not matter
    again, dagain = step(logits)
    assert all(torch.equal(want[m], again[m]) for m in want) and torch.equal(dwant, dagain)
    z = torch.zeros_like(logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, d = step(z)
    z.copy_(logits)
    graph.replay()
    assert all(torch.equal(want[m], out[m]) for m in want) and torch.equal(dwant, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, d = step(logits)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(want[m], out[m]) for m in want) and torch.equal(dwant, d)


def test_gradient_is_the_losses():
    """Differences of the fp32 loss itself along a direction: (L(z + hv) - L(z - hv)) / 2h with h = 2^-5. The losses are
    off by about 1e-6 of their size (so 2e-6 L / 2h), the difference by h^2 / 6 times the third derivative along v, which
    for v of +-1 is below 8 L: 1.4e-3 L in all."""
    T, E, k = 800, 16, 2
    for score in ("softmax", "sigmoid"):
        logits, idx, off, mask = inputs(T, E, k, torch.float32, seqs=3, pad=0.1)
        cfg = config(T, E, k, score)
        f = lambda z: rde.balance_loss(cfg, z, idx, ALPHA, off, mask)["loss"].double().sum()  # noqa: E731
        out = rde.balance_loss(cfg, logits, idx, ALPHA, off, mask)
        d = rde.balance_loss_backward(cfg, logits, out["counts"], out["tokens"], ALPHA, torch.ones(3, device="cuda"), off,
                                      mask)
        v = torch.where(d > 0, 1.0, -1.0)
        h = 2.0 ** -5
        diff = (f(logits + h * v) - f(logits - h * v)) / (2 * h)
        assert abs(float(diff) - float((d.double() * v).sum())) <= 1.5e-3 * float(f(logits))


def test_binding_refuses():
    logits, idx, off, mask = inputs(10, 8, 2, torch.float32)
    cfg = config(10, 8, 2, "softmax")
    for bad in (dict(logits=logits.T), dict(logits=logits.half()), dict(logits=logits[:5]), dict(idx=idx.long()),
                dict(mask=mask[:3]), dict(off=off.long()), dict(off=off[:1])):
        a = {**dict(logits=logits, idx=idx, off=off, mask=mask), **bad}
        with pytest.raises(ValueError):
            rde.balance_loss(cfg, a["logits"], a["idx"], ALPHA, a["off"], a["mask"])
    with pytest.raises(rde.MoeError) as e:
        rde.balance_loss(cfg, logits, idx, ALPHA, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -3
