"""Cases of the microscaled 4-bit and load-balance operators, with their plain forms.

Operators
  quantize          rows to 4-bit floating point with block scales, and the values they then stand for
  matmul            the product of two 4-bit matrices
  ffn               the experts' SwiGLU FFN on 4-bit rows and 4-bit weights, expert-major rows
  balance           the router's load-balance loss, per-expert counts and mean probabilities
  balance_backward  its gradient with respect to the router's logits

Formats: "nvfp4" has e2m1 codes, an e4m3 scale for 16 elements and one fp32 scale g for the matrix:
scale = e4m3(amax / (6 g)), code = e2m1(x / (scale * g)), each step rounded to fp32 and saturating, and
the value it stands for is code * scale * g. "mxfp4" has e2m1 codes and a power of two for 32 elements:
scale = 2^(floor(log2(amax)) - 2). Element 2i of a row is the low nibble of byte i.
"""
import math
import random

import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ALPHA = 1e-3  # weight of the balance loss
W_SIGMA = 0.02


def listed():
    return [
        # ragged rows in the power-of-two format: a small batch between two layers, latency
        {"name": "quantize ragged", "op": "quantize", "rows": 259, "cols": 2080, "fmt": "mxfp4", "type": "fp16"},
        # the rows of a prefill batch in front of a 4-bit layer
        {"name": "quantize prefill", "op": "quantize", "rows": 16384, "cols": 7168, "fmt": "nvfp4", "type": "bf16"},
        # a projection of one token: its latency
        {"name": "matmul token", "op": "matmul", "M": 1, "N": 7168, "K": 2048, "fmt": "nvfp4"},
        # odd sizes on every side, the power-of-two format
        {"name": "matmul ragged", "op": "matmul", "M": 1000, "N": 4101, "K": 2080, "fmt": "mxfp4"},
        # a projection of a prefill batch
        {"name": "matmul prefill", "op": "matmul", "M": 8192, "N": 14336, "K": 4096, "fmt": "nvfp4"},
        # few tokens through a small layer: launches and latency
        {"name": "ffn small", "op": "ffn", "T": 64, "h": 512, "I": 256, "E": 8, "k": 2, "shared": 0, "skew": 0.0,
         "fmt": "mxfp4"},
        # a decode step of a large layer with skewed experts: the weights stream from memory
        {"name": "ffn decode", "op": "ffn", "T": 256, "h": 7168, "I": 2048, "E": 256, "k": 8, "shared": 1,
         "skew": 1.2, "fmt": "nvfp4"},
        # a prefill step of the same layer: the tensor cores
        {"name": "ffn prefill", "op": "ffn", "T": 16384, "h": 7168, "I": 2048, "E": 256, "k": 8, "shared": 1,
         "skew": 0.5, "fmt": "nvfp4"},
        # a small batch of a softmax router: latency
        {"name": "balance small", "op": "balance", "T": 512, "E": 8, "k": 2, "score": "softmax", "seqs": 1,
         "pad": 0.0, "type": "fp32"},
        # a training batch of packed sequences with padding, sigmoid router, one loss per sequence
        {"name": "balance packed", "op": "balance", "T": 65536, "E": 256, "k": 8, "score": "sigmoid", "seqs": 24,
         "pad": 0.1, "type": "fp32"},
        # the gradients of two such steps
        {"name": "balance backward small", "op": "balance_backward", "T": 512, "E": 8, "k": 2, "score": "softmax",
         "seqs": 1, "pad": 0.0, "type": "bf16"},
        {"name": "balance backward packed", "op": "balance_backward", "T": 65536, "E": 256, "k": 8,
         "score": "sigmoid", "seqs": 24, "pad": 0.1, "type": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "ffn", "balance", "balance_backward"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    if op == "quantize":
        cols = 32 * _log(rng, 1, 448)
        rows = _log(rng, 1, min(65536, 16384 * 7168 // cols))
        return {"op": op, "rows": rows, "cols": cols, "fmt": fmt, "type": rng.choice(list(TYPES))}
    if op == "matmul":
        K, N = 32 * _log(rng, 1, 224), _log(rng, 1, 14336)
        return {"op": op, "M": _log(rng, 1, min(16384, 8192 * 14336 * 4096 // (N * K))), "N": N, "K": K, "fmt": fmt}
    if op == "ffn":
        E = _log(rng, 2, 256)
        h, inner = 256 * _log(rng, 1, 28), 256 * _log(rng, 1, 16)
        while E * h * inner > 256 * 7168 * 2048:
            inner = 256 * (inner // 512)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, min(16384, 16384 * 8 * 7168 * 2048 // (k * h * inner)))
        return {"op": op, "T": T, "h": h, "I": inner, "E": E, "k": k, "shared": rng.randint(0, 1),
                "skew": rng.choice([0.0, 0.5, 1.2]), "fmt": fmt}
    T, E = _log(rng, 1, 65536), _log(rng, 2, 512)
    return {"op": op, "T": T if T * E <= 65536 * 256 else 65536 * 256 // E, "E": E, "k": rng.randint(1, min(8, E)),
            "score": rng.choice(["softmax", "sigmoid"]), "seqs": _log(rng, 1, min(64, T)),
            "pad": rng.choice([0.0, 0.1, 0.5]), "type": rng.choice(["fp32", "bf16"])}


# ------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------
def _div(a, b):
    """a / b rounded once to fp32: the quotient of two fp32 numbers in 64 bits, rounded again, is that one."""
    return (a.double() / b.double()).float()


def _power(bits):
    """2^(bits - 127) in fp32."""
    bits = bits.int()
    return torch.where(bits > 0, bits << 23, 1 << 22).view(torch.float32)


def _quantize(x, fmt, g):
    """(codes [rows, cols / 2], scales [rows, cols / block]) of fp32 rows; g: fp32 tensor of one element."""
    rows, cols = x.shape
    x = x.view(rows, cols // BLOCK[fmt], BLOCK[fmt])
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        s = _div(amax, g * 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        step = s.float() * g
        bits = s.view(torch.uint8)
    else:
        # the exponent field of amax is the scale's, less 2; 2^-127 is the least one
        bits = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0).to(torch.uint8)
        step = _power(bits)
    y = torch.where(step > 0, _div(x.abs(), torch.where(step > 0, step, 1.0)), 0.0)
    # midpoints of 0, 0.5, 1, 1.5, 2, 3, 4, 6: a tie goes to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75).to(torch.uint8) + (y > 1.25).to(torch.uint8)
            + (y >= 1.75).to(torch.uint8) + (y > 2.5).to(torch.uint8) + (y >= 3.5).to(torch.uint8)
            + (y > 5.0).to(torch.uint8))
    code = (code | (torch.signbit(x) & (step > 0)).to(torch.uint8) << 3).view(rows, cols // 2, 2)
    return code[..., 0] | code[..., 1] << 4, bits.view(rows, -1)


def _values(q, s, fmt, g):
    """The fp32 values of 4-bit rows."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    grid = torch.cat((grid, -grid))
    rows, half = q.shape
    v = torch.stack((grid[(q & 15).int()], grid[(q >> 4).int()]), -1).view(rows, -1, BLOCK[fmt])
    if fmt == "nvfp4":
        v = v * s.view(torch.float8_e4m3fn).float().unsqueeze(-1)
        return v.view(rows, 2 * half) * g
    return (v * _power(s).unsqueeze(-1)).view(rows, 2 * half)


def _plain_quantize(st):
    q, s = _quantize(st["x"].float(), st["fmt"], st["g"])
    return _values(q, s, st["fmt"], st["g"])


def _plain_matmul(st):
    a, b = (_values(st[n + "q"], st[n + "s"], st["fmt"], 1.0) for n in "ab")
    return (a @ b.T * (st["ga"] * st["gb"])).to(torch.bfloat16)


def _plain_ffn(st):
    fmt, inner, y, at = st["fmt"], st["I"], [], 0
    for e, n in enumerate(st["counts"]):  # the experts' rows, then the shared expert's
        if n:
            rows = slice(at, at + n)
            x = _values(st["xq"][rows], st["xs"][rows], fmt, st["g_x"])
            gu = x @ _values(st["w_gu"][e], st["s_gu"][e], fmt, st["g_gu"][e]).T
            h = torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]
            h = _values(*_quantize(h, fmt, st["g_h"]), fmt, st["g_h"])
            o = h @ _values(st["w_d"][e], st["s_d"][e], fmt, st["g_d"][e]).T
            y.append((o * st["row_weight"][rows].unsqueeze(-1)).to(torch.bfloat16))
            at += n
    return torch.cat(y)


def _plain_probabilities(st):
    z = st["logits"].float()
    if st["score"] == "sigmoid":  # sigmoid / its sum over the experts
        z = torch.where(z > 0, -torch.log1p(torch.exp(-z.abs())), z - torch.log1p(torch.exp(-z.abs())))
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _in_sequence(st):
    """[seqs, T] truth values: the unpadded tokens of each sequence."""
    t = torch.arange(st["T"], device=st["logits"].device)
    off = st["offsets"]
    return (t >= off[:-1, None]) & (t < off[1:, None]) & st["mask"].bool()


def _plain_balance(st):
    p, ins = _plain_probabilities(st), _in_sequence(st)
    n = ins.sum(-1)
    hits = torch.zeros(st["T"], st["E"], device=p.device).scatter_(1, st["topk_idx"].long(), 1.0)
    counts = (ins.float() @ hits).round().double()  # whole numbers below 2^24: exact
    mean = (ins.double() @ p.double()) / n.clamp(min=1).unsqueeze(-1)
    loss = ALPHA * st["E"] / (st["k"] * n.clamp(min=1)) * (counts * mean).sum(-1)
    return {"loss": loss.float(), "counts": counts.int(), "mean_prob": mean.float(), "tokens": n.int()}


def _plain_balance_backward(st):
    p, ins = _plain_probabilities(st), _in_sequence(st)
    n = st["tokens"].double().clamp(min=1)
    c = (st["dloss"].double() * ALPHA * st["E"] / (st["k"] * n * n)).unsqueeze(-1) * st["counts"].double()
    g = (ins.double().T @ c).float()  # a token is in one sequence at most
    d = p * (g - (p * g).sum(-1, keepdim=True))
    if st["score"] == "sigmoid":
        d = d * torch.sigmoid(-st["logits"].float())
    return torch.where(ins.any(0).unsqueeze(-1), d, 0.0).to(st["logits"].dtype)


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _counts(case):
    """Rows of each expert, busiest first: shares that fall as 1 / rank^skew, at most one row of a token each."""
    T, E, k = case["T"], case["E"], case["k"]
    share = [(i + 1.0) ** -case["skew"] for i in range(E)]
    left, rest, out = T * k, sum(share), []
    for i in range(E):
        after = (E - i - 1) * T  # the most that later experts can take
        n = max(min(T, left, math.ceil(left * share[i] / rest)), left - after)
        out.append(n)
        left, rest = left - n, rest - share[i]
    return out


def _scale(x):
    return (x.abs().amax().float() / 2688.0).reshape(1)


def _weights(gen, n, rows, cols, fmt, dev):
    """n random matrices: (codes, scales, matrix scales)."""
    q = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(n, rows, cols // BLOCK[fmt], dtype=torch.uint8, device=dev)
    g = torch.ones(n, device=dev)
    for e in range(n):
        w = torch.randn(rows, cols, generator=gen, device=dev) * W_SIGMA
        if fmt == "nvfp4":
            g[e:e + 1] = _scale(w)
        q[e], s[e] = _quantize(w, fmt, g[e:e + 1])
    return q, s, g


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case)
    if case["op"] == "quantize":
        # activations: a few channels are much larger than the others
        chan = torch.exp(torch.randn(case["cols"], generator=gen, device=dev))
        st["x"] = (torch.randn(case["rows"], case["cols"], generator=gen, device=dev) * chan).to(TYPES[case["type"]])
        st["g"] = _scale(st["x"])
    elif case["op"] == "matmul":
        x = torch.randn(case["M"], case["K"], generator=gen, device=dev)
        st["ga"] = _scale(x) if case["fmt"] == "nvfp4" else torch.ones(1, device=dev)
        st["aq"], st["as"] = _quantize(x, case["fmt"], st["ga"])
        q, s, st["gb"] = _weights(gen, 1, case["N"], case["K"], case["fmt"], dev)
        st["bq"], st["bs"] = q[0], s[0]
    elif case["op"] == "ffn":
        T, h, inner, E, fmt = case["T"], case["h"], case["I"], case["E"], case["fmt"]
        n = E + case["shared"]
        counts = _counts(case)
        random.Random(seed).shuffle(counts)
        st["counts"] = counts + [T] * case["shared"]
        st["offsets"] = torch.tensor([0] + counts, device=dev).cumsum(0).int()
        x = torch.randn(T * case["k"] + T * case["shared"], h, generator=gen, device=dev)
        st["g_x"], st["g_h"] = torch.ones(2, 1, device=dev)
        if fmt == "nvfp4":
            st["g_x"] = _scale(x)
            st["g_h"] = torch.full((1,), 16 * W_SIGMA * W_SIGMA * h / 2688.0, device=dev)  # four sigma of gate and up
        st["xq"], st["xs"] = _quantize(x, fmt, st["g_x"])
        st["w_gu"], st["s_gu"], st["g_gu"] = _weights(gen, n, 2 * inner, h, fmt, dev)
        st["w_d"], st["s_d"], st["g_d"] = _weights(gen, n, h, inner, fmt, dev)
        st["row_weight"] = torch.rand(x.shape[0], generator=gen, device=dev)
        st["row_weight"][T * case["k"]:] = 1.0  # the shared expert's rows
        if own:
            import routing_dispatch_expert_gb300 as rde

            st["cfg"] = rde.make_config(T=T, h=h, E=E, k=case["k"], I=inner, I_shared=inner * case["shared"], dtype=fmt)
            shared = {m + "_shared": st[m][E] for m in ("w_gu", "s_gu", "w_d", "s_d")} if case["shared"] else {}
            if fmt == "nvfp4":
                shared |= {"g_gu": st["g_gu"], "g_d": st["g_d"]}
                shared |= {m + "_shared": st[m][E:].clone() for m in ("g_gu", "g_d")} if case["shared"] else {}
            st["weights"] = rde.Weights(w_router=None, w_gu=st["w_gu"], s_gu=st["s_gu"], w_d=st["w_d"], s_d=st["s_d"],
                                        **shared)
            st["act"] = rde.Fp4Activations(st["g_x"], st["g_h"]) if fmt == "nvfp4" else None
            st["ws"] = rde.alloc_workspace(st["cfg"])
            st["yd"] = torch.empty(x.shape[0], h, dtype=torch.bfloat16, device=dev)
    else:
        T, E, S = case["T"], case["E"], case["seqs"]
        skew = torch.randn(E, generator=gen, device=dev)  # some experts are liked more
        st["logits"] = (torch.randn(T, E, generator=gen, device=dev) * 1.5 + skew).to(TYPES[case["type"]])
        st["topk_idx"] = torch.topk(st["logits"].float(), case["k"], -1).indices.int()
        cuts = torch.rand(S - 1, generator=gen, device=dev).sort().values * T
        st["offsets"] = torch.cat((cuts.new_zeros(1), cuts, cuts.new_full((1,), T))).int()
        st["mask"] = (torch.rand(T, generator=gen, device=dev) >= case["pad"]).to(torch.uint8)
        if case["op"] == "balance_backward":
            out = _plain_balance(st)
            st["counts"], st["tokens"] = out["counts"], out["tokens"]
            st["dloss"] = 1.0 + torch.rand(S, generator=gen, device=dev)
        if own:
            import routing_dispatch_expert_gb300 as rde

            st["cfg"] = rde.make_config(T=T, h=256, E=E, k=case["k"], I=256, score=case["score"])
            st["ws"] = rde.balance_loss_workspace(st["cfg"], S)
    return st


def run(st):
    if not own:
        return {"quantize": _plain_quantize, "matmul": _plain_matmul, "ffn": _plain_ffn, "balance": _plain_balance,
                "balance_backward": _plain_balance_backward}[st["op"]](st)
    import routing_dispatch_expert_gb300 as rde

    if st["op"] == "quantize":
        g = st["g"] if st["fmt"] == "nvfp4" else None
        q, s = rde.quantize_fp4(st["x"], st["fmt"], g)
        return rde.dequantize_fp4(q, s, st["fmt"], g)
    if st["op"] == "matmul":
        scales = {"ga": st["ga"], "gb": st["gb"]} if st["fmt"] == "nvfp4" else {}
        return rde.matmul_fp4(st["aq"], st["as"], st["bq"], st["bs"], st["fmt"], **scales)
    if st["op"] == "ffn":
        rde.expert_ffn_fp4(st["cfg"], st["weights"], st["act"], st["xq"], st["xs"], st["offsets"], st["row_weight"],
                           st["yd"], st["ws"])
        return st["yd"]
    if st["op"] == "balance":
        return rde.balance_loss(st["cfg"], st["logits"], st["topk_idx"], ALPHA, seq_offsets=st["offsets"],
                                token_mask=st["mask"], ws=st["ws"])
    return rde.balance_loss_backward(st["cfg"], st["logits"], st["counts"], st["tokens"], ALPHA, st["dloss"],
                                     seq_offsets=st["offsets"], token_mask=st["mask"])


def work(case):
    if case["op"] in ("quantize", "matmul", "ffn"):
        bits4 = 0.5 + 1.0 / BLOCK[case["fmt"]]  # bytes of an element and its share of the scale
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]  # rows in, codes and scales out, values out
        return {"bytes": int(n * (TYPES[case["type"]].itemsize + bits4 + 4)), "flops": 2 * n}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": int((M + N) * K * bits4 + 2 * M * N), "flops": 2 * M * N * K}
    if case["op"] == "ffn":
        T, h, inner = case["T"], case["h"], case["I"]
        rows = T * (case["k"] + case["shared"])
        active = sum(n > 0 for n in _counts(case)) + case["shared"]
        return {"bytes": int(active * 3 * h * inner * bits4 + rows * (h * bits4 + 2 * h + 4)),
                "flops": 6 * rows * h * inner}
    T, E = case["T"], case["E"]
    b = TYPES[case["type"]].itemsize
    if case["op"] == "balance":
        return {"bytes": T * (E * b + 4 * case["k"] + 1) + case["seqs"] * E * 8, "flops": 6 * T * E}
    return {"bytes": T * (2 * E * b + 1) + case["seqs"] * E * 4, "flops": 8 * T * E}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _exp2(e):
    """2^e for whole e, without rounding."""
    return torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)[e.long() + 200]


def _round_to(v, least, mantissa, most):
    """Magnitudes v (fp64) to the nearest number of a small float type, ties to even, saturating."""
    v = v.clamp(max=most)
    _, e = torch.frexp(v.clamp(min=least))
    step = _exp2(e - 1 - mantissa)
    return torch.round(v / step) * step


def _exact_values(x, fmt, g):
    """What the fp64 rows x stand for in 4 bits; g: a number. The format itself rounds to fp32 on the way."""
    rows, cols = x.shape
    x = x.view(rows, -1, BLOCK[fmt])
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        six = torch.tensor(g * 6.0, device=x.device).float().double()
        s = _round_to((amax / six).float().double(), 2.0 ** -6, 3, 448.0)
        step = (s * g).float().double()
    else:
        _, e = torch.frexp(amax)
        s = _exp2(torch.where(amax > 0, e - 3, -127).clamp(min=-127))
        step, g = s, 1.0
    y = torch.where(step > 0, (x / step).float().double(), 0.0)
    return (torch.sign(y) * _round_to(y.abs(), 1.0, 1, 6.0) * s * g).view(rows, cols)


def _exact_decode(q, s, fmt, g):
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2).double()
    sign = torch.where(code >= 8, -1.0, 1.0).double()
    m = code % 8
    v = torch.where(m < 2, m / 2, (1 + m % 2 / 2) * _exp2(torch.floor(m / 2) - 1)) * sign
    if fmt == "nvfp4":
        b = s.double()
        scale = torch.where(b < 8, b / 512, (1 + b % 8 / 8) * _exp2(torch.floor(b / 8) - 7)) * g
    else:
        scale = _exp2(s.double() - 127)
    return v * scale.repeat_interleave(BLOCK[fmt], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(st["x"].double(), st["fmt"], float(st["g"]))
    if op == "matmul":
        if case["M"] * case["N"] * case["K"] > 2e12:
            return None
        a = _exact_decode(st["aq"], st["as"], st["fmt"], float(st["ga"]))
        return a @ _exact_decode(st["bq"], st["bs"], st["fmt"], float(st["gb"])).T
    if op == "ffn":
        if work(case)["flops"] > 2e12:
            return None
        y, at, fmt, inner = [], 0, st["fmt"], st["I"]
        for e, n in ((e, n) for e, n in enumerate(st["counts"]) if n):
            rows = slice(at, at + n)
            x = _exact_decode(st["xq"][rows], st["xs"][rows], fmt, float(st["g_x"]))
            gate, up = (x @ _exact_decode(st["w_gu"][e], st["s_gu"][e], fmt, float(st["g_gu"][e])).T).split(inner, 1)
            h = _exact_values(gate / (1 + torch.exp(-gate)) * up, fmt, float(st["g_h"]))
            o = h @ _exact_decode(st["w_d"][e], st["s_d"][e], fmt, float(st["g_d"][e])).T
            y.append(o * st["row_weight"][rows].double().unsqueeze(1))
            at += n
        return torch.cat(y)
    z = st["logits"].double()
    s = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
    p = s / s.sum(-1, keepdim=True)
    seq = torch.bucketize(torch.arange(case["T"], device=z.device), st["offsets"][1:].long(), right=True)
    seq = torch.where(st["mask"].bool(), seq, case["seqs"])  # padding: a sequence of its own, left out
    n = torch.bincount(seq, minlength=case["seqs"] + 1)[:-1]
    S, E, k = case["seqs"], case["E"], case["k"]
    at = (seq.unsqueeze(1) * E + st["topk_idx"].long()).flatten()
    counts = torch.bincount(at, minlength=(S + 1) * E).view(S + 1, E)[:-1].double()
    f = torch.where(n > 0, ALPHA * E / (k * n.double()), 0.0)
    if op == "balance":
        mean = torch.zeros(S + 1, E, dtype=torch.float64, device=z.device).index_add_(0, seq, p)[:-1]
        mean = mean / n.clamp(min=1).unsqueeze(1)
        return {"loss": f * (counts * mean).sum(-1), "counts": None, "mean_prob": mean, "tokens": None}
    g = torch.cat((st["dloss"].double() * torch.where(n > 0, f / n, 0.0), z.new_zeros(1))).unsqueeze(1)
    g = (g * torch.cat((counts, z.new_zeros(1, E))))[seq]
    d = p * (g - (p * g).sum(-1, keepdim=True))
    return d * (1 - s) if case["score"] == "sigmoid" else d
