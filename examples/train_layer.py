"""Trains a small mixture-of-experts layer: norm, router, experts, and the residual stream around them.

The library's operators, each with its gradient, carry the tokens: the norm of the residual stream (rms_norm), the route
weights (route_weights) and the load-balance loss (balance_loss) of the router's logits, the tokens sorted by expert
(sort_tokens), their rows into that order (permute) and back, weighted and added to the stream (unpermute). The experts
themselves are torch products here, one expert after the other.

    python examples/train_layer.py [--steps 20]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import routing_dispatch_expert_gb300 as rde  # noqa: E402


class Layer(torch.nn.Module):
    def __init__(self, h, E, k, I, score="softmax", capacity_factor=0.0):
        super().__init__()
        self.shape = dict(h=h, E=E, k=k, I=I, score=score, renorm=True, capacity_factor=capacity_factor)
        self.norm = torch.nn.Parameter(torch.ones(h))
        self.router = torch.nn.Parameter(torch.randn(E, h) * h ** -0.5)
        self.gate_up = torch.nn.Parameter(torch.randn(E, 2 * I, h) * h ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(E, h, I) * I ** -0.5)

    def forward(self, x, alpha=0.01):
        """(stream after the layer, balance loss) of the stream x [T, h]."""
        cfg = rde.make_config(T=x.shape[0], **self.shape)
        y = rde.rms_norm(x, self.norm)
        logits = y.float() @ self.router.T
        idx, weights = rde.route_weights(cfg, logits)
        balance = rde.balance_loss(cfg, logits, idx, alpha)["loss"].sum()
        s = rde.sort_tokens(cfg, idx)
        rows = rde.permute(cfg, y, s["inv_pos"], s["offsets"])
        parts, bounds = [], s["offsets"].tolist()
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            gate, up = (rows[lo:hi] @ self.gate_up[e].to(rows.dtype).T).chunk(2, -1)
            parts.append((torch.nn.functional.silu(gate) * up) @ self.down[e].to(rows.dtype).T)
        parts.append(rows[bounds[-1]:])  # rows that hold nothing (a capacity limit): zeros
        out = rde.unpermute(cfg, torch.cat(parts), s["inv_pos"], weights, base=x, offsets=s["offsets"])
        return out, balance


def main(steps=20, T=2048, h=256, E=16, k=2, I=128, dtype=torch.bfloat16, lr=3e-3):
    torch.manual_seed(0)
    x = torch.randn(T, h, device="cuda")
    target = x + torch.tanh(x @ torch.randn(h, h, device="cuda") * h ** -0.5)
    layer = Layer(h, E, k, I).cuda()
    optimizer = torch.optim.Adam(layer.parameters(), lr=lr)
    history = []
    for step in range(steps + 1):
        out, balance = layer(x.to(dtype))
        loss = torch.nn.functional.mse_loss(out.float(), target)
        optimizer.zero_grad(set_to_none=True)
        (loss + balance).backward()
        optimizer.step()
        history.append((float(loss.detach()), float(balance.detach())))
        if step % 5 == 0 or step == steps:
            print(f"step {step:3d}: loss {history[-1][0]:.4f}, balance loss {history[-1][1]:.5f}")
    return history, layer


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=20)
    main(p.parse_args().steps)
