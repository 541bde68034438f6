"""A layer of experts on the library's operators: a few training steps in
bf16, then the trained layer in fp8 and in 4 bits on a prompt, and in fp8 token
by token.

    python examples/expert_layer.py [--tokens 2048] [--hidden 1024] [--inner 512]
                                    [--experts 16] [--top 2] [--steps 20]

Each row is normalised and goes to its `top` best experts; an expert is
    y = W_down (silu(W_gate x) * W_up x)
with the gate and up products as one.  The tokens are sorted by expert once and
copied into that order, the grouped products take the group boundaries from the
device, and the weighted sums return to the tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from communication_gemm_amd.experts import (  # noqa: E402
    combine, dispatch, grouped_linear, grouped_linear_fp8, grouped_linear_mxfp4, quantize_mxfp4,
    quantize_weights, rms_norm, rms_norm_fp8, sort_by_expert)


class Experts(torch.nn.Module):
    def __init__(self, hidden, inner, experts, top):
        super().__init__()
        self.top, self.inner = top, inner
        make = lambda *s: torch.nn.Parameter(  # noqa: E731
            torch.randn(*s, device="cuda", dtype=torch.bfloat16) * s[-2] ** -0.5)
        self.norm = torch.nn.Parameter(torch.ones(hidden, device="cuda", dtype=torch.bfloat16))
        self.router = make(hidden, experts)
        self.w_in = make(experts, hidden, 2 * inner)     # gate and up, side by side
        self.w_out = make(experts, inner, hidden)

    def route(self, x):
        """Each token's weights, and where its copies go."""
        weight, chosen = torch.softmax((x @ self.router).float(), -1).topk(self.top, -1)
        return weight, sort_by_expert(chosen, self.router.shape[1])

    def activate(self, h):
        return torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]

    def forward(self, x):
        x = rms_norm(x, self.norm)
        weight, r = self.route(x)
        h = self.activate(grouped_linear(dispatch(x, r), self.w_in, r.offsets))
        return combine(grouped_linear(h, self.w_out, r.offsets), weight, r)

    @torch.no_grad()
    def to_low_bits(self):
        """Weights as the fp8 and 4-bit products take them: [E, out, in]."""
        w = [t.transpose(1, 2).contiguous() for t in (self.w_in, self.w_out)]
        self.fp8 = [quantize_weights(t) for t in w]      # scales of 128 x 128
        self.mxfp4 = [quantize_mxfp4(t) for t in w]      # and of 1 x 32

    @torch.no_grad()
    def serve_fp8(self, x):
        q, scale, x = rms_norm_fp8(x, self.norm, with_y=True)
        weight, r = self.route(x)
        rows = dispatch(q, r), dispatch(scale, r)
        h = self.activate(grouped_linear_fp8(rows, *self.fp8[0], r.offsets, x.dtype))
        return combine(grouped_linear_fp8(h, *self.fp8[1], r.offsets), weight, r)

    @torch.no_grad()
    def serve_mxfp4(self, x):
        x = rms_norm(x, self.norm)
        weight, r = self.route(x)
        h = self.activate(grouped_linear_mxfp4(dispatch(x, r), *self.mxfp4[0], r.offsets))
        return combine(grouped_linear_mxfp4(h, *self.mxfp4[1], r.offsets), weight, r)


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
    layer.to_low_bits()
    with torch.no_grad():
        full, fp8, mxfp4 = (f(x).float() for f in (layer, layer.serve_fp8, layer.serve_mxfp4))
        one = torch.cat([layer.serve_fp8(x[i:i + 1]) for i in range(8)]).float()
    off, off4 = (((t - full).norm() / full.norm()).item() for t in (fp8, mxfp4))
    print("against bf16: fp8 %.3f of the norm, 4 bits %.3f; one token at a time against the prompt: %.4f" % (
        off, off4, ((one - fp8[:8]).norm() / fp8[:8].norm()).item()))
    return losses, off


if __name__ == "__main__":
    main()
