"""Rebalances the router of a layer whose experts are frozen in 4 bits.

Every step runs the layer with 4-bit rows and weights (moe_forward_fp4), takes the load-balance loss of its routing
and the per-expert counts (moe_balance_loss), and moves the router's fp32 weight against the loss's gradient
(moe_balance_loss_backward): the experts, the routing and the loss are the library's, the weight's own gradient is
one product, dlogits^T x.

    python examples/rebalance_router_fp4.py [--steps 30] [--format nvfp4|mxfp4]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import routing_dispatch_expert_gb300 as rde  # noqa: E402


def quantized_weights(w_router, w_gu, w_d, fmt):
    """The layer's weights with the experts [E, rows, cols] in 4 bits."""
    t = {"w_router": w_router}
    for name, w in (("gu", w_gu), ("d", w_d)):
        if fmt == "nvfp4":
            t["w_" + name], t["s_" + name], t["g_" + name] = rde.quantize_weights_nvfp4(w)
        else:
            q, s = rde.quantize_fp4(w.view(-1, w.shape[-1]), fmt)
            t["w_" + name], t["s_" + name] = (v.view(*w.shape[:2], -1) for v in (q, s))
    return rde.Weights(**t)


def calibrate(x, w_gu, fmt):
    """Activation scales from the largest magnitudes that a sample of rows brings about."""
    if fmt == "mxfp4":
        return rde.Fp4Activations()
    gate, up = (x[:256].float() @ w_gu[:4].float().mT).chunk(2, -1)
    h = torch.nn.functional.silu(gate) * up
    return rde.Fp4Activations(*(v.abs().amax().float().reshape(1) / 2688 for v in (x, h)))


def main(steps=30, fmt="nvfp4", T=4096, h=512, E=32, k=4, I=256, alpha=1.0, lr=0.01, seqs=8):
    torch.manual_seed(0)
    dev = "cuda"
    w_gu = (torch.randn(E, 2 * I, h, device=dev) * 0.05).to(torch.bfloat16)
    w_d = (torch.randn(E, h, I, device=dev) * 0.05).to(torch.bfloat16)
    liked = torch.randn(E, 1, device=dev) * 0.015  # some experts' scores share a direction with every token
    mean = torch.randn(h, device=dev) * 0.5
    w_router = torch.randn(E, h, device=dev) * 0.02 + liked * mean
    x = (torch.randn(T, h, device=dev) + mean).to(torch.bfloat16)
    bounds = torch.arange(seqs + 1, device=dev, dtype=torch.int32) * (T // seqs)

    cfg = rde.make_config(T=T, h=h, E=E, k=k, I=I, score="softmax", renorm=True, dtype=fmt)
    weights = quantized_weights(w_router, w_gu, w_d, fmt)
    layer = rde.MoeLayer(cfg, weights, fp4_activations=calibrate(x, w_gu, fmt))
    ws = rde.balance_loss_workspace(cfg, seqs)
    y = torch.empty_like(x)
    dloss = torch.full((seqs,), 1.0 / seqs, device=dev)  # the mean over the sequences
    history = []
    for step in range(steps + 1):
        layer(x, y)
        logits = rde.ws_view(layer.ws, cfg, "logits", torch.float32, (T, E))
        chosen = rde.ws_view(layer.ws, cfg, "topk_idx", torch.int32, (T, k))
        out = rde.balance_loss(cfg, logits, chosen, alpha, seq_offsets=bounds, ws=ws)
        dlogits = rde.balance_loss_backward(cfg, logits, out["counts"], out["tokens"], alpha, dloss, seq_offsets=bounds)
        w_router -= lr * (dlogits.T @ x.float())
        if step % 5 == 0 or step == steps:
            load = rde.balance(cfg, layer.ws)
            history.append((float(out["loss"].mean()), load["max_over_mean"]))
            print(f"step {step:3d}: balance loss {history[-1][0]:.4f}, busiest expert {history[-1][1]:.2f} x the mean")
    if rde.device_status(cfg, layer.ws):
        raise RuntimeError("the layer reported bad data or a timed-out wait")
    return history, y


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    a = p.parse_args()
    main(a.steps, a.format)
