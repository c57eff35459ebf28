"""Cases of the operators around the experts that training and 8-bit serving need, with their plain forms.

Operators
  norm                root-mean-square norm of x + residual, also as e4m3 codes with a scale for 128 elements
  norm_backward       its gradient
  permute             tokens sorted by expert, and their rows copied into that order
  unpermute           the rows back in token order, weighted and added (without weights: permute's gradient)
  unpermute_backward  its gradient with respect to the rows and the weights
  route_backward      gradient of the route weights with respect to the router's logits

Rows of an expert are in the order of their assignments (token, then slot). An expert index outside [0, E) is no
assignment (padding); with a capacity factor an expert keeps the first ceil(factor T k / E). What is not assigned or not
kept has position -1 and no row; rows behind the last one are zero, with token -1 and weight 0.
Codes in 8 bits are returned as float8 values, next to their scales: scale = amax / 448 of 128 elements, at least 2^-126
(1 where all are zero), code = value / scale.
"""
import math
import random

import torch

own = False

EPS = 1e-6
SCALE = 2.5  # routed scaling factor
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # the norm in front of a layer for one token: latency
        {"name": "norm token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "residual": "bf16",
         "weight": "bf16", "fp8": False},
        # a prefill batch in front of a router and an 8-bit layer, the residual stream carried on
        {"name": "norm fp8 prefill", "op": "norm", "rows": 16384, "cols": 7168, "type": "bf16", "residual": "bf16",
         "weight": "bf16", "fp8": True},
        # a small ragged batch in full precision: odd rows, no gradient from the residual stream
        {"name": "norm backward ragged", "op": "norm_backward", "rows": 1000, "cols": 4101, "type": "fp32",
         "total": "fp32", "weight": "fp32", "dtotal": False},
        # a training batch
        {"name": "norm backward prefill", "op": "norm_backward", "rows": 16384, "cols": 7168, "type": "bf16",
         "total": "bf16", "weight": "fp32", "dtotal": True},
        # a decode step of a large layer: the sort's latency
        {"name": "permute decode", "op": "permute", "T": 256, "cols": 7168, "E": 256, "k": 8, "type": "bf16",
         "pad": 0.0, "cap": 0.0},
        # a prefill batch whose rows are 8-bit already
        {"name": "permute fp8 prefill", "op": "permute", "T": 16384, "cols": 7168, "E": 256, "k": 8, "type": "e4m3",
         "pad": 0.0, "cap": 0.0},
        # few tokens of a small layer: latency
        {"name": "unpermute small", "op": "unpermute", "T": 64, "cols": 512, "E": 8, "k": 2, "type": "bf16",
         "pad": 0.0, "cap": 0.0, "weighted": True, "base": False},
        # a prefill batch, weighted and added to the residual stream
        {"name": "unpermute prefill", "op": "unpermute", "T": 16384, "cols": 7168, "E": 256, "k": 8, "type": "bf16",
         "pad": 0.0, "cap": 0.0, "weighted": True, "base": True},
        # odd rows, padded tokens, a capacity limit
        {"name": "unpermute backward ragged", "op": "unpermute_backward", "T": 999, "cols": 1003, "E": 60, "k": 6,
         "type": "fp16", "pad": 0.1, "cap": 1.25},
        # a training batch
        {"name": "unpermute backward prefill", "op": "unpermute_backward", "T": 16384, "cols": 7168, "E": 256, "k": 8,
         "type": "bf16", "pad": 0.0, "cap": 0.0},
        # a small softmax router
        {"name": "route backward small", "op": "route_backward", "T": 4096, "E": 8, "k": 2, "score": "softmax",
         "renorm": False, "pad": 0.0, "type": "fp32"},
        # a large sigmoid router whose weights are normalised
        {"name": "route backward large", "op": "route_backward", "T": 65536, "E": 256, "k": 8, "score": "sigmoid",
         "renorm": True, "pad": 0.05, "type": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cols(rng, least=1):
    n = _log(rng, least, 8192)
    return n if rng.random() < 0.4 else min(8192, 64 * -(-n // 64))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "permute", "unpermute", "unpermute_backward", "route_backward"])
    kind = rng.choice(["bf16", "fp16", "fp32"])
    size = TYPES[kind].itemsize
    if op in ("norm", "norm_backward"):
        cols = _cols(rng, 1 if op == "norm" else 8)  # in rows of a few numbers the gradient cancels
        rows = _log(rng, 1, min(65536, 16384 * 7168 * 2 // (cols * size)))
        total = rng.choice([kind, kind, "fp32"])
        case = {"op": op, "rows": rows, "cols": cols, "type": kind, "weight": rng.choice([kind, "fp32", "none"])}
        if op == "norm":
            return case | {"residual": rng.choice([total, total, "none"]), "fp8": rng.random() < 0.5}
        return case | {"total": total, "dtotal": rng.random() < 0.5}
    E = _log(rng, 2, 1024)
    k = rng.randint(1, min(8, E))
    pad = rng.choice([0.0, 0.1, 0.5])
    if op == "route_backward":
        return {"op": op, "T": _log(rng, 1, min(65536, 65536 * 256 // E)), "E": E, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "pad": pad,
                "renorm": k > 1 and rng.random() < 0.5,  # one normalised weight does not change
                "type": rng.choice(["fp32", "bf16"])}
    if op == "permute":
        kind = rng.choice(["bf16", "fp32", "e4m3"])
    cols = _cols(rng)
    T = _log(rng, 1, min(65536, 16384 * 8 * 7168 * (1 if op == "permute" else 2) // (cols * k * TYPES[kind].itemsize)))
    case = {"op": op, "T": T, "cols": cols, "E": E, "k": k, "type": kind, "pad": pad, "cap": rng.choice([0.0, 1.25])}
    if op == "unpermute":
        case |= {"weighted": rng.random() < 0.6, "base": rng.random() < 0.5}
    return case


# ------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------
def _blocks(n):
    return -(-n // 128)


def _quantize(y):
    """(codes, scales) of fp32 rows."""
    rows, cols = y.shape
    n = _blocks(cols)
    y = torch.nn.functional.pad(y, (0, 128 * n - cols)).view(rows, n, 128)
    amax = y.abs().amax(-1)
    s = torch.where(amax > 0, (amax / 448.0).clamp(min=2.0 ** -126), 1.0)
    q = (y / s.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(rows, 128 * n)[:, :cols], s


def _plain_norm(st):
    total = st["x"].float()
    if st["r"] is not None:
        total = total + st["r"].float()
    y = total * torch.rsqrt((total * total).mean(-1, keepdim=True) + EPS)
    if st["w"] is not None:
        y = y * st["w"].float()
    out = {"y": y.to(st["x"].dtype)}
    if st["r"] is not None:
        out["total"] = total.to(st["r"].dtype)
    if st["fp8"]:
        out["q"], out["s"] = _quantize(y)
    return out


def _plain_norm_backward(st):
    t, g = st["t"].float(), st["dy"].float()
    rstd = torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)
    n = t * rstd
    per_weight = g * n
    if st["w"] is not None:
        g = g * st["w"].float()
    d = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if st["dt"] is not None:
        d = d + st["dt"].float()
    out = {"dx": d.to(st["dy"].dtype)}
    if st["t"].dtype != st["dy"].dtype:
        out["dresidual"] = d.to(st["t"].dtype)
    if st["w"] is not None:
        out["dweight"] = per_weight.sum(0, dtype=torch.float64).to(st["w"].dtype)
    return out


def _capacity(case):
    n = case["T"] * case["k"]
    return math.ceil(case["cap"] * case["T"] * case["k"] / case["E"]) if case["cap"] else n


def _plain_sort(idx, weight, E, capacity):
    T, k = idx.shape
    n, dev = T * k, idx.device
    e = idx.flatten().long()
    e = torch.where((e >= 0) & (e < E), e, E)
    key, order = torch.sort(e, stable=True)
    every = torch.zeros(E + 1, dtype=torch.long, device=dev).scatter_add_(0, e, torch.ones_like(e))
    first = every.cumsum(0) - every
    rank = torch.arange(n, device=dev) - first[key]
    counts = every[:E].clamp(max=capacity)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    row = torch.where((key < E) & (rank < capacity), offsets[key] + rank, n)  # n: no row
    inv = torch.empty_like(e).scatter_(0, order, row)
    token = torch.full((n + 1,), -1, dtype=torch.long, device=dev).scatter_(0, row, order // k)[:n]
    w = torch.zeros(n + 1, device=dev).scatter_(0, row, weight.flatten()[order])[:n]
    inv = torch.where(inv < n, inv, -1).view(T, k)
    held = torch.arange(n, device=dev) < offsets[E]
    return {"counts": counts.int(), "offsets": offsets.int(), "inv_pos": inv.int(),
            "row_token": torch.where(held, token, -1).int(), "row_weight": torch.where(held, w, 0.0)}


def _rows(x, row_token):
    """Rows of x, zero where there is none; 8-bit rows are moved as bytes."""
    b = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    b = torch.where((row_token >= 0).unsqueeze(-1), b[row_token.clamp(min=0).long()], torch.zeros((), dtype=b.dtype, device=b.device))
    return b.view(x.dtype)


def _plain_permute(st):
    out = _plain_sort(st["idx"], st["weights"], st["E"], st["capacity"])
    out["xd"] = _rows(st["x"], out["row_token"])
    if st["s"] is not None:
        out["xd_scales"] = _rows(st["s"], out["row_token"])
    return out


def _plain_unpermute(st):
    inv = st["inv_pos"]
    rows = st["yd"][inv.clamp(min=0).flatten().long()].view(*inv.shape, -1).float()
    rows = torch.where((inv >= 0).unsqueeze(-1), rows, 0.0)
    if st["weighted"]:
        rows = rows * st["weights"].unsqueeze(-1)
    y = rows.sum(1)
    if st["b"] is not None:
        y = y + st["b"].float()
    return y.to(st["yd"].dtype)


def _plain_unpermute_backward(st):
    inv, token = st["inv_pos"], st["row_token"]
    held = (token >= 0).unsqueeze(-1)
    dy = torch.where(held, st["dy"][token.clamp(min=0).long()], 0.0).float()
    dots = (torch.where(held, st["yd"], 0.0).float() * dy).sum(-1)
    dw = torch.where(inv >= 0, dots[inv.clamp(min=0).long()], 0.0)
    return {"dyd": (dy * st["row_weight"].unsqueeze(-1)).to(st["yd"].dtype), "dweights": dw}


def _plain_route_backward(st):
    z, idx, g = st["logits"].float(), st["idx"], st["dweights"]
    chosen = (idx >= 0) & (idx < st["E"])
    at = torch.where(chosen, idx, 0).long()
    g = torch.where(chosen, g, 0.0)
    l = torch.where(chosen, z.gather(1, at), -math.inf)
    if st["score"] == "softmax" and not st["renorm"]:
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        p = p / p.sum(-1, keepdim=True)
        dense = torch.zeros_like(z).scatter_add_(1, at, g)
        return (SCALE * p * (dense - (p * dense).sum(-1, keepdim=True))).to(st["logits"].dtype)
    if st["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True).clamp(min=-1e30))
        u = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
        d = u * (g - (u * g).sum(-1, keepdim=True))
    else:
        s, c = torch.sigmoid(l), torch.sigmoid(-l)
        if st["renorm"]:
            u = s / s.sum(-1, keepdim=True).clamp(min=1e-30)
            d = u * c * (g - (u * g).sum(-1, keepdim=True))
        else:
            d = s * c * g
    return torch.zeros_like(z).scatter_add_(1, at, torch.where(chosen, SCALE * d, 0.0)).to(st["logits"].dtype)


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _route(case, gen, dev):
    """(logits, chosen experts, weights): some experts are liked more, and padded tokens choose none."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=gen, device=dev) * 1.5 + torch.randn(E, generator=gen, device=dev)
    idx = torch.topk(logits, k, -1).indices.int()
    idx = torch.where(torch.rand(T, 1, generator=gen, device=dev) < case["pad"], -1, idx).int()
    w = torch.rand(T, k, generator=gen, device=dev) + 0.05
    return logits, idx, SCALE * w / w.sum(-1, keepdim=True)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case)

    def rows(n, kind, scale=1.0):
        if kind == "none":
            return None
        return (torch.randn(n, case["cols"], generator=gen, device=dev) * scale).to(TYPES[kind])

    if case["op"] in ("norm", "norm_backward"):
        chan = torch.exp(0.5 * torch.randn(case["cols"], generator=gen, device=dev))  # some channels are larger
        st["w"] = None
        if case["weight"] != "none":
            st["w"] = (1.0 + 0.2 * torch.randn(case["cols"], generator=gen, device=dev)).to(TYPES[case["weight"]])
        if case["op"] == "norm":
            st["x"], st["r"] = rows(case["rows"], case["type"]), rows(case["rows"], case["residual"], 2.0 * chan)
        else:
            st["t"], st["dy"] = rows(case["rows"], case["total"], 2.0 * chan), rows(case["rows"], case["type"], 0.01)
            st["dt"] = rows(case["rows"], case["total"], 0.01) if case["dtotal"] else None
        return st
    st["logits"], st["idx"], st["weights"] = _route(case, gen, dev)
    if case["op"] == "route_backward":
        st["logits"] = st["logits"].to(TYPES[case["type"]])
        st["dweights"] = torch.randn(case["T"], case["k"], generator=gen, device=dev)
    else:
        st["capacity"] = _capacity(case)
        if case["op"] == "permute":
            st["x"], st["s"] = rows(case["T"], "fp32" if case["type"] == "e4m3" else case["type"]), None
            if case["type"] == "e4m3":
                st["x"], st["s"] = _quantize(st["x"])
                st["x"] = st["x"].contiguous()
        else:  # the state that the forward pass left
            st |= _plain_sort(st["idx"], st["weights"], case["E"], st["capacity"])
            st["yd"] = rows(case["T"] * case["k"], case["type"])
            if case["op"] == "unpermute":
                st["b"] = rows(case["T"], case["type"], 2.0) if case["base"] else None
            else:
                st["dy"] = rows(case["T"], case["type"], 0.01)
    if own:
        import routing_dispatch_expert_gb300 as rde

        st["cfg"] = rde.make_config(T=case["T"], h=256, E=case["E"], k=case["k"], I=256, capacity_factor=case.get("cap", 0.0),
                                    score=case.get("score", "softmax"), renorm=case.get("renorm", False),
                                    routed_scale=SCALE)
    return st


def run(st):
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "permute": _plain_permute,
                "unpermute": _plain_unpermute, "unpermute_backward": _plain_unpermute_backward,
                "route_backward": _plain_route_backward}[st["op"]](st)
    import routing_dispatch_expert_gb300 as rde

    if st["op"] == "norm":
        if st["fp8"]:
            out = rde.rms_norm_fp8(st["x"], st["w"], residual=st["r"], eps=EPS, with_y=True)
            out["q"] = out["q"].view(torch.float8_e4m3fn)
            return out
        if st["r"] is None:
            return {"y": rde.rms_norm(st["x"], st["w"], eps=EPS)}
        y, total = rde.rms_norm(st["x"], st["w"], residual=st["r"], eps=EPS)
        return {"y": y, "total": total}
    if st["op"] == "norm_backward":
        out = rde.rms_norm_backward(st["dy"], st["t"], st["w"], eps=EPS, dtotal=st["dt"])
        return {"dx": out[0], **({"dresidual": out[1]} if out[1] is not out[0] else {}),
                **({} if st["w"] is None else {"dweight": out[2]})}
    if st["op"] == "permute":
        out = rde.sort_tokens(st["cfg"], st["idx"], st["weights"])
        if st["s"] is None:
            out["xd"] = rde.permute(st["cfg"], st["x"], out["inv_pos"], out["offsets"])
        else:
            q, out["xd_scales"] = rde.permute(st["cfg"], st["x"].view(torch.uint8), out["inv_pos"], out["offsets"],
                                              scales=st["s"])
            out["xd"] = q.view(torch.float8_e4m3fn)
        return out
    if st["op"] == "unpermute":
        return rde.unpermute(st["cfg"], st["yd"], st["inv_pos"], st["weights"] if st["weighted"] else None, base=st["b"])
    if st["op"] == "unpermute_backward":
        dyd, dw = rde.unpermute_backward(st["cfg"], st["dy"], st["yd"], st["inv_pos"], st["offsets"], st["weights"])
        return {"dyd": dyd, "dweights": dw}
    return rde.route_backward(st["cfg"], st["logits"], st["idx"], st["dweights"])


def work(case):
    op = case["op"]
    size = TYPES[case["type"]].itemsize
    if op in ("norm", "norm_backward"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        wide = lambda kind: 0 if kind == "none" else TYPES[kind].itemsize  # noqa: E731
        w = cols * wide(case["weight"])
        if op == "norm":  # x, residual and weight in, their sum, y and the codes out
            b = n * (2 * size + 2 * wide(case["residual"])) + w
            if case["fp8"]:
                b += n + 4 * case["rows"] * _blocks(cols)
            return {"bytes": b, "flops": 5 * n}
        t = wide(case["total"])  # dy, total and its gradient in, one gradient of each type out
        b = n * (2 * size + t + (t if case["dtotal"] else 0) + (t if case["total"] != case["type"] else 0)) + 2 * w
        return {"bytes": b, "flops": 12 * n}
    T, k, E = case["T"], case["k"], case["E"]
    if op == "route_backward":
        dense = case["score"] == "softmax" and not case["renorm"]  # needs every logit, the others the chosen ones
        return {"bytes": T * (E * size + (E if dense else k) * size + 8 * k), "flops": T * (4 * E if dense else E + 8 * k)}
    cols, rows = case["cols"], int(T * k * (1 - case["pad"]))
    if op == "permute":
        b = size * cols + (4 * _blocks(cols) if case["type"] == "e4m3" else 0)
        return {"bytes": (T + rows) * b + T * k * 20 + 8 * E, "flops": T * k}
    if op == "unpermute":
        return {"bytes": size * cols * (rows + T * (1 + case["base"])) + T * k * (8 if case["weighted"] else 4),
                "flops": 2 * rows * cols}
    return {"bytes": size * cols * (2 * rows + T) + T * k * 12, "flops": 3 * rows * cols}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_norm(st):
    x = st["x"].double()
    t = x if st["r"] is None else x + st["r"].double()
    y = t / torch.sqrt(t.pow(2).mean(1, keepdim=True) + EPS)
    if st["w"] is not None:
        y.mul_(st["w"].double())
    out = {"y": y}
    if st["r"] is not None:
        out["total"] = t
    if st["fp8"]:
        m, c, n = *y.shape, _blocks(y.shape[1])
        big = torch.zeros(m, 128 * n, dtype=torch.float64, device=y.device)
        big[:, :c] = y
        s = big.view(m, n, 128).abs().max(-1).values / 448
        s = torch.where(s == 0, 1.0, s.clamp(min=2.0 ** -126))
        out["s"], out["q"] = s, y / s.repeat_interleave(128, 1)[:, :c]  # before the rounding to 8 bits
    return out


def _exact_norm_backward(st):
    t, dy = st["t"].double(), st["dy"].double()
    m = t.pow(2).mean(1, keepdim=True) + EPS
    w = 1.0 if st["w"] is None else st["w"].double()
    d = dy * w / m.sqrt() - t * ((dy * w * t).mean(1, keepdim=True) / m.pow(1.5))
    if st["dt"] is not None:
        d += st["dt"].double()
    out = {"dx": d}
    if st["t"].dtype != st["dy"].dtype:
        out["dresidual"] = d
    if st["w"] is not None:
        out["dweight"] = (dy * t / m.sqrt()).sum(0)
    return out


def _exact_permute(st):
    """Each expert's assignments, one expert after the other."""
    e, T, k = st["idx"].flatten(), *st["idx"].shape
    keep = [torch.nonzero(e == i).squeeze(1)[:st["capacity"]] for i in torch.unique(e[(e >= 0) & (e < st["E"])]).tolist()]
    at = torch.cat(keep) if keep else torch.empty(0, dtype=torch.long, device=e.device)
    n = at.numel()
    out = {"counts": None, "offsets": None, "inv_pos": None, "row_token": None}
    for name, v in (("xd", st["x"]), ("xd_scales", st["s"]), ("row_weight", st["weights"])):
        if v is not None:
            v = v.double()
            out[name] = v.new_zeros(T * k, *v.shape[1:]) if name != "row_weight" else v.new_zeros(T * k)
            out[name][:n] = v[at // k] if name != "row_weight" else v.flatten()[at]
    return out


def _exact_unpermute(st):
    inv = st["inv_pos"].long()
    y = torch.zeros(inv.shape[0], st["yd"].shape[1], dtype=torch.float64, device=inv.device)
    if st["b"] is not None:
        y += st["b"].double()
    for j in range(inv.shape[1]):
        t = torch.nonzero(inv[:, j] >= 0).squeeze(1)
        rows = st["yd"][inv[t, j]].double()
        y[t] += rows * st["weights"][t, j].double().unsqueeze(1) if st["weighted"] else rows
    return y


def _exact_unpermute_backward(st):
    inv, w = st["inv_pos"].long(), st["weights"].double()
    dyd = torch.zeros(st["yd"].shape, dtype=torch.float64, device=inv.device)
    dw = torch.zeros_like(w)
    for j in range(inv.shape[1]):
        t = torch.nonzero(inv[:, j] >= 0).squeeze(1)
        dy = st["dy"][t].double()
        dyd[inv[t, j]] = dy * w[t, j].unsqueeze(1)
        dw[t, j] = (st["yd"][inv[t, j]].double() * dy).sum(1)
    return {"dyd": dyd, "dweights": dw}


def _exact_route_backward(st):
    """By the chain rule from each chosen weight, one after the other."""
    z = st["logits"].double()
    T, E = z.shape
    one = torch.nn.functional.one_hot(torch.where((st["idx"] < 0) | (st["idx"] >= E), E, st["idx"]).long(), E + 1)
    one = one[..., :E].double()  # [T, k, E]
    g = st["dweights"].double() * SCALE
    if st["score"] == "softmax":
        v, slope = torch.exp(z - z.max(1, keepdim=True).values), 1.0
    else:
        v, slope = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))  # d v / d z = v * slope
    picked = torch.einsum("tke,te->tk", one, v)
    if st["renorm"] or st["score"] == "softmax":
        total = picked.sum(1, keepdim=True) if st["renorm"] else v.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        # d (v_j / total) = d v_j / total - v_j / total^2 * d total
        shared = (g * picked).sum(1, keepdim=True) / total ** 2
        dv = torch.einsum("tke,tk->te", one, g) / total - shared * (one.sum(1) if st["renorm"] else 1.0)
    else:
        dv = torch.einsum("tke,tk->te", one, g)
    return dv * v * slope


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "permute": _exact_permute,
            "unpermute": _exact_unpermute, "unpermute_backward": _exact_unpermute_backward,
            "route_backward": _exact_route_backward}[case["op"]](st)
