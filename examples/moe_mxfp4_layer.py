"""A mixture-of-experts layer with 4-bit experts: trained straight through, then served.

The layer is router -> permute -> up projection -> SiLU -> down projection -> weighted un-permute. Its
experts multiply in MXFP4: the fp32 master weights are quantised once per training step, the activations
where they enter a projection. The backward pass differentiates through the quantised operands as if
quantisation were the identity (straight-through): it multiplies by the bf16 values the codes stand
for, and reaches the experts, the token rows and the router's gate. Serving keeps the codes and scales
alone and takes one token at a time.

    python examples/moe_mxfp4_layer.py --steps 60
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import group_gemm_gb300 as gg  # noqa: E402

ROUTER = "softmax_topk"


class MoeLayer:
    """fp32 master weights: gate [dim, E], up [E, dim, hidden], down [E, hidden, dim]."""

    def __init__(self, dim, hidden, experts, topk, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=gen, device=device) * shape[-2] ** -0.5
        self.topk, self.experts = topk, experts
        self.gate, self.up, self.down = rand(dim, experts), rand(experts, dim, hidden), rand(experts, hidden, dim)
        self.quantise()

    def parameters(self):
        return {"gate": self.gate, "up": self.up, "down": self.down}

    def quantise(self):
        """Lays the experts out for the 4-bit products; call it after the master weights change."""
        self.up_q, self.up_s, self.up_v = gg.quantize_mxfp4_weight(self.up, values=True)
        self.down_q, self.down_s, self.down_v = gg.quantize_mxfp4_weight(self.down, values=True)

    def forward(self, x, keep=False):
        """x bf16 [T, dim] -> bf16 [T, dim]; with ``keep`` also what :meth:`backward` needs."""
        logits = x.float() @ self.gate
        ids, w = gg.router_topk(logits, self.topk, ROUTER)
        xs, sizes, order, inv = gg.moe_permute(ids, x, self.experts)
        xq, xscale, *xv = gg.quantize_mxfp4(xs, values=keep)
        h = gg.ragged_dot_mxfp4(xq, xscale, self.up_q, self.up_s, sizes)
        act = torch.nn.functional.silu(h)
        aq, ascale, *av = gg.quantize_mxfp4(act, values=keep)
        y = gg.ragged_dot_mxfp4(aq, ascale, self.down_q, self.down_s, sizes)
        out = gg.moe_unpermute(y, inv, w)
        if not keep:
            return out
        return out, (x, logits, ids, w, sizes, order, inv, xv[0], h, av[0], y)

    def backward(self, dout, kept):
        """The gradients of the weights and of x for the output's gradient dout (bf16 [T, dim])."""
        x, logits, ids, w, sizes, order, inv, xv, h, av, y = kept
        dy, dw = gg.moe_unpermute_grad(dout, y, order, inv, w)
        d_down = gg.grad_weight(av, dy, sizes)
        dact = gg.grad_input(dy, self.down_v, sizes)
        hf = h.float()
        sig = torch.sigmoid(hf)
        dh = (dact.float() * sig * (1 + hf * (1 - sig))).to(torch.bfloat16)
        d_up = gg.grad_weight(xv, dh, sizes)
        dx = gg.moe_permute_grad(gg.grad_input(dh, self.up_v, sizes), inv, self.topk)
        dlogits = gg.router_topk_grad(logits, ids, w, dw, ROUTER)
        dx = dx.float() + dlogits @ self.gate.t()
        return {"gate": x.float().t() @ dlogits, "up": d_up, "down": d_down}, dx


def train(layer, teacher, steps, tokens, dim, device, lr=0.02, seed=1):
    """Fits the layer to a fixed teacher's outputs with Adam; returns the losses."""
    gen = torch.Generator(device=device).manual_seed(seed)
    moments = {n: (torch.zeros_like(p), torch.zeros_like(p)) for n, p in layer.parameters().items()}
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn((tokens, dim), generator=gen, device=device).to(torch.bfloat16)
        target = teacher(x)
        out, kept = layer.forward(x, keep=True)
        err = out.float() - target
        losses.append(float((err * err).mean()))
        grads, _ = layer.backward((2.0 / err.numel() * err).to(torch.bfloat16), kept)
        for name, p in layer.parameters().items():
            m, v = moments[name]
            m.mul_(0.9).add_(grads[name], alpha=0.1)
            v.mul_(0.99).addcmul_(grads[name], grads[name], value=0.01)
            p.sub_(lr * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-12))
        layer.quantise()
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2)
    args = ap.parse_args(argv)
    device = torch.device("cuda", torch.cuda.current_device())
    gg.build()

    gen = torch.Generator(device=device).manual_seed(7)
    mix = torch.randn((args.dim, args.dim), generator=gen, device=device) * args.dim ** -0.5
    layer = MoeLayer(args.dim, args.hidden, args.experts, args.topk, device)
    losses = train(layer, lambda x: torch.tanh(x.float() @ mix), args.steps, args.tokens, args.dim, device)
    print(f"training loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")

    # serving: the same codes, a batch at once and token by token
    x = torch.randn((8, args.dim), generator=gen, device=device).to(torch.bfloat16)
    batch = layer.forward(x)
    single = torch.cat([layer.forward(x[i:i + 1]) for i in range(len(x))])
    print(f"8 tokens at once and one by one differ by at most {float((batch.float() - single.float()).abs().max()):.2e}")
    return losses, batch, single


if __name__ == "__main__":
    main()
