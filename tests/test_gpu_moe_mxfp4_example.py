"""The 4-bit layer example on the GPU: its gradients against autograd of the same layer in 64 bits on
the quantised values, and the training and serving run it shows."""
import os
import sys

import pytest
import torch

import group_gemm_gb300 as gg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    gg.build()
    gg.load()
    import moe_mxfp4_layer
    return moe_mxfp4_layer


def test_layer_gradients_against_autograd(example):
    dim, hidden, experts, topk, tokens = 128, 192, 5, 2, 77
    layer = example.MoeLayer(dim, hidden, experts, topk, DEV, seed=3)
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((tokens, dim), generator=gen, device=DEV).to(torch.bfloat16)
    out, kept = layer.forward(x, keep=True)
    dout = torch.randn(out.shape, generator=gen, device=DEV).to(torch.bfloat16)
    grads, dx = layer.backward(dout, kept)
    ids = kept[2].long()

    # the same layer in 64 bits; quantisation is the identity for the gradient, so each quantised operand
    # is its value plus (operand - operand detached)
    def through(value, operand):
        return value.double() + operand - operand.detach()

    gate = layer.gate.double().requires_grad_()
    up, down = layer.up.double().requires_grad_(), layer.down.double().requires_grad_()
    x64 = x.double().requires_grad_()
    w = torch.softmax((x64 @ gate).gather(1, ids), 1)
    sel = ids.reshape(-1)
    flat = kept[6].long()                                  # sorted row of each copy
    xin = through(kept[7][flat], x64.repeat_interleave(topk, 0))
    h = torch.einsum("ck,ckn->cn", xin, through(layer.up_v, up)[sel])
    act = torch.nn.functional.silu(h)
    y = torch.einsum("ck,ckn->cn", through(kept[9][flat], act), through(layer.down_v, down)[sel])
    ref = (w.unsqueeze(-1) * y.view(tokens, topk, dim)).sum(1)
    ref.backward(dout.double())
    # each stored bf16 intermediate (dy, dact, dh, dxs, y, h, out) is off by at most 2^-8 of itself, with
    # either sign: seven of them bound the relative 2-norm by 7 * 2^-8
    tol = 7 * 2.0 ** -8
    for name, got, want in (("out", out, ref), ("gate", grads["gate"], gate.grad), ("up", grads["up"], up.grad),
                            ("down", grads["down"], down.grad), ("x", dx, x64.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= tol, (name, rel)


def test_example_trains_and_serves(example):
    losses, batch, single = example.main(["--steps", "40", "--tokens", "256", "--dim", "128", "--hidden", "256"])
    assert losses[-1] < 0.7 * losses[0]
    # one token takes the same codes through the same products: equal up to the order of fp32 sums and the
    # roundings to bf16 that follow (h, y and the output: three half steps of the largest output)
    assert float((batch.float() - single.float()).abs().max()) <= 3 * 2.0 ** -8 * float(batch.float().abs().max())
