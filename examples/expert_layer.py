"""A layer of experts on the grouped products: a few training steps in
bf16, then the trained layer in fp8 on a prompt and token by token.

    python examples/expert_layer.py [--tokens 2048] [--hidden 1024] [--inner 512]
                                    [--experts 16] [--top 2] [--steps 20]

Each token goes to its `top` best experts; an expert is
    y = W_down (silu(W_gate x) * W_up x)
with the gate and up products as one.  The rows are sorted by expert once
(an argsort of the chosen experts), the grouped products take the group
boundaries from the device, and the weighted sums return to the tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from communication_gemm_amd.experts import (  # noqa: E402
    grouped_linear, grouped_linear_fp8, quantize_weights)


class Experts(torch.nn.Module):
    def __init__(self, hidden, inner, experts, top):
        super().__init__()
        self.top, self.inner = top, inner
        make = lambda *s: torch.nn.Parameter(  # noqa: E731
            torch.randn(*s, device="cuda", dtype=torch.bfloat16) * s[-2] ** -0.5)
        self.router = make(hidden, experts)
        self.w_in = make(experts, hidden, 2 * inner)     # gate and up, side by side
        self.w_out = make(experts, inner, hidden)

    def route(self, x):
        """The (token, expert) pairs sorted by expert: tokens, offsets, weights."""
        weight, chosen = torch.softmax((x @ self.router).float(), -1).topk(self.top, -1)
        order = torch.argsort(chosen.flatten(), stable=True)
        counts = torch.bincount(chosen.flatten(), minlength=self.router.shape[1])
        offsets = torch.zeros(len(counts) + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = counts.cumsum(0)
        return order // self.top, offsets, weight.flatten()[order]

    def activate(self, h):
        return torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]

    def combine(self, x, tokens, y, weight):
        return torch.zeros_like(x, dtype=torch.float32).index_add(
            0, tokens, y.float() * weight[:, None]).to(x.dtype)

    def forward(self, x):
        tokens, offsets, weight = self.route(x)
        h = self.activate(grouped_linear(x[tokens], self.w_in, offsets))
        return self.combine(x, tokens, grouped_linear(h, self.w_out, offsets), weight)

    @torch.no_grad()
    def to_fp8(self):
        """Weights as the fp8 products take them: [E, out, in], 128 x 128 scales."""
        self.q_in = quantize_weights(self.w_in.transpose(1, 2).contiguous())
        self.q_out = quantize_weights(self.w_out.transpose(1, 2).contiguous())

    @torch.no_grad()
    def serve(self, x):
        tokens, offsets, weight = self.route(x)
        h = self.activate(grouped_linear_fp8(x[tokens], *self.q_in, offsets))
        return self.combine(x, tokens, grouped_linear_fp8(h, *self.q_out, offsets), weight)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 2048), ("hidden", 1024), ("inner", 512), ("experts", 16),
                        ("top", 2), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    torch.manual_seed(0)
    layer = Experts(a.hidden, a.inner, a.experts, a.top)
    teacher = Experts(a.hidden, a.inner, a.experts, a.top)
    opt = torch.optim.Adam(layer.parameters(), lr=1e-3)
    losses = []
    x = torch.randn(a.tokens, a.hidden, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        target = teacher(x)
    for _ in range(a.steps):
        loss = (layer(x) - target).float().square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print("training loss %.4f -> %.4f" % (losses[0], losses[-1]))
    layer.to_fp8()
    with torch.no_grad():
        full, fp8 = layer(x).float(), layer.serve(x).float()
        one = torch.cat([layer.serve(x[i:i + 1]) for i in range(8)]).float()
    off = ((fp8 - full).norm() / full.norm()).item()
    print("fp8 against bf16: %.3f of the norm; one token at a time against the prompt: %.4f" % (
        off, ((one - fp8[:8]).norm() / fp8[:8].norm()).item()))
    return losses, off


if __name__ == "__main__":
    main()
