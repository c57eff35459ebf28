"""Microscaled 4-bit formats and the balance loss in 64 bits, from their definitions. Test infrastructure only."""
from __future__ import annotations

import torch

BLOCK = {"nvfp4": 16, "mxfp4": 32}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# every e4m3 number from 0 to 448 by its code
E4M3 = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)],
                    dtype=torch.float64)


def nearest(values, v):
    """Index of the nearest of the ascending numbers `values` to each v >= 0; ties to the even index; saturating."""
    values = values.to(v.device)
    mids = (values[1:] + values[:-1]) / 2
    lo = torch.bucketize(v, mids)  # mids < v
    tie = torch.isin(v, mids) & (lo % 2 == 1)
    return lo + tie


def scale_values(s, fmt):
    s = s.long()
    if fmt == "nvfp4":
        table = torch.cat((E4M3, torch.full((1,), float("nan"), dtype=torch.float64)))
        return table.to(s.device)[s & 127]
    table = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [float("nan")], dtype=torch.float64)
    return table.to(s.device)[s]


def code_values(q):
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    v = GRID.to(q.device)[c & 7]
    return torch.where(c > 7, -v, v)


def values(q, s, fmt, g=1.0):
    """fp64 values of 4-bit rows."""
    return code_values(q) * scale_values(s, fmt).repeat_interleave(BLOCK[fmt], -1) * g


def quantize(x, fmt, g=1.0):
    """(codes, scales) of rows; x any float type; g a python float holding an fp32 number."""
    rows, cols = x.shape
    x = x.double()
    b = x.view(rows, cols // BLOCK[fmt], BLOCK[fmt])
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad.unsqueeze(-1), 0.0, b)
    amax = b.abs().amax(-1)
    r32 = lambda t: t.float().double()  # noqa: E731
    if fmt == "nvfp4":
        six = r32(torch.tensor(6.0 * g, dtype=torch.float64)).to(x.device)
        s = nearest(E4M3, r32(amax / six))
        step = r32(E4M3.to(x.device)[s] * g)
        nan = 0x7F
    else:
        e = torch.frexp(amax)[1] - 1  # floor(log2)
        s = torch.where(amax > 0, e + 125, 0).clamp(min=0)
        step = scale_values(s, fmt)
        nan = 0xFF
    y = torch.where(step.unsqueeze(-1) > 0, r32(b / torch.where(step > 0, step, 1.0).unsqueeze(-1)), 0.0)
    code = nearest(GRID, y.abs())
    code = code + 8 * (torch.signbit(b) & (step > 0).unsqueeze(-1) & ~bad.unsqueeze(-1))
    code = code.view(rows, cols // 2, 2).to(torch.uint8)
    s = torch.where(bad, nan, s).to(torch.uint8)
    return code[..., 0] | code[..., 1] << 4, s


def silu(v):
    return v / (1 + torch.exp(-v))


def probabilities(logits, score):
    z = logits.double()
    if score == "sigmoid":
        z = torch.nn.functional.logsigmoid(z)  # normalised sigmoids: a softmax of their logarithms
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isneginf(m), 0.0, m)
    e = torch.exp(z - m)
    t = e.sum(-1, keepdim=True)
    return torch.where(t == 0, 0.0, e / t)


def balance_loss(logits, topk_idx, score, alpha, offsets=None, mask=None):
    """Per sequence, one after the other: dict as routing_dispatch_expert_gb300.balance_loss, in fp64."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    offsets = [0, T] if offsets is None else [int(v) for v in offsets]
    mask = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask.bool()
    out = {"loss": [], "counts": [], "mean_prob": [], "tokens": []}
    for a, b in zip(offsets[:-1], offsets[1:]):
        rows = torch.arange(a, b, device=logits.device)
        rows = rows[mask[rows]]
        n = rows.numel()
        idx = topk_idx[rows].flatten().long()
        counts = torch.bincount(idx[(idx >= 0) & (idx < E)], minlength=E)
        mean = probabilities(logits[rows], score).mean(0) if n else torch.zeros(E, dtype=torch.float64,
                                                                                device=logits.device)
        out["loss"].append((alpha * E / (k * n) * (counts.double() * mean).sum()) if n else mean.sum())
        out["counts"].append(counts)
        out["mean_prob"].append(mean)
        out["tokens"].append(torch.tensor(n))
    return {m: torch.stack(v) for m, v in out.items()}


def balance_loss_backward(logits, counts, k, score, alpha, dloss, offsets=None, mask=None):
    """d (dloss . loss) / d logits in fp64, from the formula."""
    T, E = logits.shape
    offsets = [0, T] if offsets is None else [int(v) for v in offsets]
    mask = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask.bool()
    d = torch.zeros(T, E, dtype=torch.float64, device=logits.device)
    for s, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        rows = torch.arange(a, b, device=logits.device)
        rows = rows[mask[rows]]
        n = rows.numel()
        if n == 0:
            continue
        p = probabilities(logits[rows], score)
        c = counts[s].double()
        g = float(dloss[s]) * alpha * E / (k * n * n) * p * (c - (p * c).sum(-1, keepdim=True))
        if score == "sigmoid":
            g = g * torch.sigmoid(-logits[rows].double())
        d[rows] = g
    return d
