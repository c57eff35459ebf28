"""Definitions in 64 bits of the norm, the row permutation and the gradients: what the tests compare with. Plain torch,
any device. Test infrastructure only."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}  # of a rounding, relative
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half the least number


def norm(x, weight, residual, eps):
    """(y, total) in 64 bits."""
    t = x.double() if residual is None else x.double() + residual.double()
    y = t / torch.sqrt(t.pow(2).mean(1, keepdim=True) + eps)
    return (y if weight is None else y * weight.double()), t


def norm_backward(dy, total, weight, eps, dtotal=None):
    """(gradient of the total, of the weight, and the sums of magnitudes that their errors are relative to)."""
    t, dy = total.double(), dy.double()
    rstd = 1 / torch.sqrt(t.pow(2).mean(1, keepdim=True) + eps)
    g = dy if weight is None else dy * weight.double()
    n = t * rstd
    d = rstd * (g - n * (g * n).mean(1, keepdim=True))
    size = rstd * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dtotal is not None:
        d = d + dtotal.double()
        size = size + dtotal.double().abs()
    return d, (dy * n).sum(0), size, (dy * n).abs().sum(0)


def sort(idx, E, capacity=None, placement=None):
    """Python loops: (counts, offsets, inv_pos, row_token, row of weights' flat index or -1). placement: the plan's
    arrays as lists (slot_expert, slot_replica, replicas, replica_slot)."""
    T, k = idx.shape
    flat = idx.flatten().tolist()
    of = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E and (capacity is None or len(of[e]) < capacity):
            of[e].append(i)
    if placement is None:
        groups = of
    else:
        groups = [of[e][r::placement["replicas"][e]] for e, r in zip(placement["slot_expert"], placement["slot_replica"])]
    counts = [len(g) for g in groups]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    order = [i for g in groups for i in g]
    inv = [-1] * (T * k)
    for row, i in enumerate(order):
        inv[i] = row
    source = order + [-1] * (T * k - len(order))
    return {"counts": counts, "offsets": offsets, "inv_pos": inv, "row_token": [i // k if i >= 0 else -1 for i in source],
            "source": source}


def unpermute(yd, inv_pos, weights, base):
    """(y, sum of magnitudes) in 64 bits."""
    T, k = inv_pos.shape
    inv = inv_pos.long()
    rows = torch.where((inv >= 0).unsqueeze(-1), yd[inv.clamp(min=0)].double(), 0.0)
    if weights is not None:
        rows = rows * torch.where(inv >= 0, weights.double(), 0.0).unsqueeze(-1)
    y, size = rows.sum(1), rows.abs().sum(1)
    return (y, size) if base is None else (y + base.double(), size + base.double().abs())


def unpermute_backward(dy, yd, inv_pos, weights):
    """(dyd, dweights, sum of magnitudes of dweights) in 64 bits."""
    inv = inv_pos.long()
    dyd = torch.zeros(yd.shape, dtype=torch.float64, device=yd.device)
    dw = torch.zeros(inv.shape, dtype=torch.float64, device=yd.device)
    size = torch.zeros_like(dw)
    for j in range(inv.shape[1]):
        t = torch.nonzero(inv[:, j] >= 0).squeeze(1)
        w = 1.0 if weights is None else weights[t, j].double().unsqueeze(1)
        dyd[inv[t, j]] = w * dy[t].double()
        p = yd[inv[t, j]].double() * dy[t].double()
        dw[t, j], size[t, j] = p.sum(1), p.abs().sum(1)
    return dyd, dw, size


def route_weights(logits, idx, score, renorm, scale):
    """The weights of chosen experts in 64 bits (0 for an index outside the experts)."""
    T, E = logits.shape
    ok = (idx >= 0) & (idx < E)
    z = logits.double()
    l = z.gather(1, torch.where(ok, idx, 0).long())
    if score == "softmax":
        m = z.amax(1, keepdim=True) if not renorm else torch.where(ok, l, -math.inf).amax(1, keepdim=True)
        v = torch.exp(l - m)
        total = torch.exp(z - m).sum(1, keepdim=True)
    else:
        v, total = 1 / (1 + torch.exp(-l)), 1.0
    v = torch.where(ok, v, 0.0)
    if renorm:
        total = v.sum(1, keepdim=True)
    return scale * torch.where(ok, v / total, 0.0)


def route_backward(logits, idx, dw, score, renorm, scale):
    """(gradient, sum of magnitudes) in 64 bits, slot by slot from the derivative of each weight."""
    T, E = logits.shape
    z = logits.double()
    ok = (idx >= 0) & (idx < E)
    out, size = torch.zeros_like(z), torch.zeros_like(z)
    for t in range(T):
        slots = [(int(idx[t, j]), float(dw[t, j])) for j in range(idx.shape[1]) if ok[t, j]]
        s = torch.softmax(z[t], 0) if score == "softmax" else torch.sigmoid(z[t])
        slope = s if score == "softmax" else s * torch.sigmoid(-z[t])  # d v / d l, v the unnormalised score
        if renorm:
            total = sum(float(s[e]) for e, _ in slots)
            dot = sum(g * float(s[e]) for e, g in slots) / total if slots else 0.0
            mag = sum(abs(g) * float(s[e]) for e, g in slots) / total if slots else 0.0
            for e, g in slots:
                out[t, e] += scale * slope[e] / total * (g - dot)
                size[t, e] += scale * slope[e] / total * (abs(g) + mag)
        elif score == "softmax":
            dot, mag = (sum(f(g) * float(s[e]) for e, g in slots) for f in (float, abs))
            out[t] -= scale * s * dot
            size[t] += scale * s * mag
            for e, g in slots:
                out[t, e] += scale * s[e] * g
                size[t, e] += scale * s[e] * abs(g)
        else:
            for e, g in slots:
                out[t, e] += scale * slope[e] * g
                size[t, e] += scale * slope[e] * abs(g)
    return out, size
