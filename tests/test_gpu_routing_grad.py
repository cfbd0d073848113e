"""GPU parity of the routing gradients (un-permute, permute, router top-k) with plain 64-bit forms of
the same formulas on the same inputs, and with differences of the 64-bit forward.

Tolerances follow from the arithmetic. u = 2^-24 is an fp32 rounding relative to the value, and a
rounding to bf16 is off by at most 2^-8 of it. A sum of n fp32 terms added in any order is off by at
most n u times the sum of their magnitudes.
"""
import pytest
import torch

import group_gemm_gb300 as gg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TINY = 2.0 ** -126      # below this a result may be subnormal: absolute steps


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def close(got, ref, tol):
    """|got - ref| <= tol element by element (tol: a float64 tensor or number)."""
    err = (got.double() - ref).abs()
    bad = ~(err <= tol + TINY)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float((err - tol).max()):.3g} over"


def routing(tokens, topk, experts, drop, seed, n=16):
    """ids with dropped copies, and the permute's own outputs for them."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.rand((tokens, experts), generator=gen, device=DEV).argsort(1)[:, :topk].int()
    if topk > experts:
        ids = torch.randint(0, experts, (tokens, topk), generator=gen, device=DEV).int()
    ids[torch.rand(ids.shape, generator=gen, device=DEV) < drop] = -1
    x = torch.randn((tokens, n), generator=gen, device=DEV).to(torch.bfloat16)
    xs, gs, order, inv = gg.moe_permute(ids, x, experts)
    return gen, order, inv, int(gs.sum())


def unpermute_ref(dout, y, order, inv, w):
    t, k = w.shape
    d, w64 = dout.double(), w.double()
    kept = inv >= 0
    yi = torch.where(kept.unsqueeze(1), y[inv.clamp(min=0).long()].double(), 0.0).view(t, k, -1)
    prod = yi * d.unsqueeze(1)
    dw, mag = prod.sum(-1), prod.abs().sum(-1)
    f = order.clamp(min=0).long()
    dy = torch.where((order >= 0).unsqueeze(1), w64.reshape(-1)[f].unsqueeze(1) * d[f // k], 0.0)
    return dy, dw, mag


CASES = [          # tokens, topk, experts, n, share of dropped copies
    (1, 1, 1, 8, 0.0), (1, 2, 8, 64, 0.0), (1, 8, 256, 7168, 0.2), (3, 2, 8, 264, 0.0), (33, 4, 5, 1032, 0.3),
    (257, 8, 128, 4096, 0.1), (700, 1, 3, 24, 0.0), (64, 40, 7, 136, 0.1), (50, 3, 4, 512, 1.0),
    (5000, 2, 8, 128, 0.05), (701, 1, 3, 24, 0.1), (1001, 3, 64, 512, 0.1), (333, 5, 9, 2048, 0.0),
]


@pytest.mark.parametrize("tokens,topk,experts,n,drop", CASES)
def test_unpermute_grad(tokens, topk, experts, n, drop):
    gen, order, inv, valid = routing(tokens, topk, experts, drop, 1)
    dout = torch.randn((tokens, n), generator=gen, device=DEV).to(torch.bfloat16)
    y = torch.randn((tokens * topk, n), generator=gen, device=DEV).to(torch.bfloat16)
    w = torch.randn((tokens, topk), generator=gen, device=DEV)
    y[valid:] = float("nan")                               # rows no copy is sorted to are never read
    w = torch.where((inv >= 0).view(tokens, topk), w, float("nan"))   # nor weights of dropped copies
    dy, dw = gg.moe_unpermute_grad(dout, y, order, inv, w)
    ref_dy, ref_dw, mag = unpermute_ref(dout, y, order, inv, w)
    # dy: one fp32 product, one rounding to bf16. dw: n products summed in fp32
    close(dy, ref_dy, (2.0 ** -8 + 2 * U) * ref_dy.abs())
    close(dw, ref_dw, n * U * mag)
    assert torch.all(dy[valid:] == 0)
    assert torch.all(dw.view(-1)[inv < 0] == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,topk,experts,n,drop", CASES)
def test_permute_grad(tokens, topk, experts, n, drop, dtype):
    gen, order, inv, valid = routing(tokens, topk, experts, drop, 2)
    dxs = torch.randn((tokens * topk, n), generator=gen, device=DEV).to(dtype)
    dxs[valid:] = float("nan")
    dx = gg.moe_permute_grad(dxs, inv, topk)
    rows = torch.where((inv >= 0).unsqueeze(1), dxs[inv.clamp(min=0).long()].double(), 0.0).view(tokens, topk, n)
    ref = rows.sum(1)
    close(dx, ref, topk * U * rows.abs().sum(1) + HALF[dtype] * ref.abs())
    if drop == 1.0:
        assert torch.all(dx == 0)


def router_ref(logits, ids, w, g, mode):
    l64, w64, g64 = logits.double(), w.double(), g.double()
    out = torch.zeros_like(l64)
    if mode == "values":
        return out.scatter(1, ids.long(), g64), out
    s = (w64 * g64).sum(1, keepdim=True)
    if mode == "softmax_topk":
        return out.scatter(1, ids.long(), w64 * (g64 - s)), out
    p = torch.softmax(l64, 1)
    return out.scatter(1, ids.long(), w64 * g64) - p * s, p


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", ["values", "softmax", "softmax_topk"])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 8, 2), (37, 33, 5), (300, 256, 8), (17, 1000, 32),
                                              (5, 1024, 1), (4097, 8, 2), (9, 32, 32)])
def test_router_topk_grad(tokens, experts, k, mode, dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    logits = (3 * torch.randn((tokens, experts), generator=gen, device=DEV)).to(dtype)
    ids, w = gg.router_topk(logits, k, mode)
    g = torch.randn((tokens, k), generator=gen, device=DEV)
    dl = gg.router_topk_grad(logits, ids, w, g, mode)
    assert dl.dtype == dtype and dl.shape == logits.shape
    ref, p = router_ref(logits, ids, w, g, mode)
    # terms w (g - s): s sums k products; p: expf (2 steps) of an argument off by u |x - m|, over a sum
    # of `experts` of them, and the product with s
    wg = (w.double() * g.double()).abs().sum(1, keepdim=True)
    spread = (logits.double().amax(1, keepdim=True) - logits.double().amin(1, keepdim=True))
    tol = (k + 8) * U * (wg + wg.new_zeros(ref.shape).scatter(1, ids.long(), (w.double() * g.double()).abs()))
    if mode == "softmax":
        tol = tol + p * wg * U * (2 * (4 + spread) + experts + k + 8)
    close(dl, ref, tol + (HALF[dtype] + U) * ref.abs())


def test_router_topk_grad_of_special_logits():
    """A row with -inf logits has zero gradient there; a NaN logit (whose weights are NaN) a NaN row in
    softmax mode; the other modes only touch the selected experts."""
    logits = torch.zeros((3, 8), device=DEV)
    logits[0, 2:] = float("-inf")
    logits[1, 5] = float("nan")
    for mode in ("values", "softmax", "softmax_topk"):
        ids, w = gg.router_topk(logits, 2, mode)
        dl = gg.router_topk_grad(logits, ids, w, torch.tensor([[1.0, -2.0]] * 3, device=DEV), mode)
        assert torch.all(dl[0, 2:] == 0) and torch.isfinite(dl[0]).all() and torch.isfinite(dl[2]).all()
        assert torch.isnan(dl[1]).all() if mode == "softmax" else torch.isfinite(dl[1]).all()


def test_router_topk_grad_counts_bad_and_repeated_ids():
    """An id outside the experts counts as none (its weight still enters the softmax's sum); copies of one
    expert, which the router never makes, add up."""
    for experts in (8, 40, 300):
        logits = torch.randn((3, experts), generator=torch.Generator(device=DEV).manual_seed(9), device=DEV)
        ids = torch.tensor([[1, -1, 5], [7, 7, 7], [experts, 0, 6]], dtype=torch.int32, device=DEV)
        w = torch.tensor([[0.5, 0.25, 0.25]] * 3, device=DEV)
        g = torch.tensor([[1.0, 2.0, -3.0]] * 3, device=DEV)
        for mode in ("values", "softmax_topk"):
            term = g if mode == "values" else w * (g - (w * g).sum(1, keepdim=True))
            want = torch.zeros((3, experts), device=DEV)
            for t in range(3):
                for j in range(3):
                    if 0 <= ids[t, j] < experts:
                        want[t, ids[t, j]] += term[t, j]
            assert torch.equal(gg.router_topk_grad(logits, ids, w, g, mode), want)


def test_gradients_agree_with_differences_of_the_forward():
    """The whole routed sum L = <c, sum_j w_j(logits) (x_sorted * a)[inv]> in 64 bits: its central
    differences along random directions against the gradients chained through the three kernels."""
    tokens, topk, experts, n = 40, 3, 9, 64
    gen = torch.Generator(device=DEV).manual_seed(5)
    logits = torch.randn((tokens, experts), generator=gen, device=DEV)
    x = torch.randn((tokens, n), generator=gen, device=DEV).to(torch.bfloat16)
    a = torch.randn((tokens * topk, n), generator=gen, device=DEV).double()
    c = torch.randn((tokens, n), generator=gen, device=DEV).to(torch.bfloat16)
    for mode in ("softmax", "softmax_topk", "values"):
        ids, w = gg.router_topk(logits, topk, mode)
        xs, gs, order, inv = gg.moe_permute(ids, x, experts)

        def weights(l):
            sel = l.gather(1, ids.long())
            return {"values": sel, "softmax_topk": torch.softmax(sel, 1),
                    "softmax": torch.softmax(l, 1).gather(1, ids.long())}[mode]

        def loss(x64, l64):
            y = x64[(order // topk).long()] * a
            return (weights(l64).unsqueeze(-1) * y[inv.long()].view(tokens, topk, n) * c.double().unsqueeze(1)).sum()

        y = (x.double()[(order // topk).long()] * a).to(torch.bfloat16)
        dy, dw = gg.moe_unpermute_grad(c, y, order, inv, w)
        dx = gg.moe_permute_grad((dy.double() * a).float(), inv, topk)
        dl = gg.router_topk_grad(logits, ids, w, dw, mode)
        for which, grad, base in (("x", dx, x.double()), ("logits", dl, logits.double())):
            u = torch.randn(base.shape, generator=gen, device=DEV).double()
            eps = 1e-4
            up, down = [(loss(base + s * eps * u, logits.double()) if which == "x" else loss(x.double(), base + s * eps * u))
                        for s in (1, -1)]
            diff, along = float((up - down) / (2 * eps)), float((grad.double() * u).sum())
            # y and dy carry one bf16 rounding per element, with random signs
            scale = float((grad.double() * u).norm())
            assert abs(diff - along) <= 8 * 2.0 ** -8 * scale + 1e-6 * abs(diff), (mode, which, diff, along, scale)


def test_expanded_and_strided_inputs_and_a_stream():
    tokens, topk, n = 30, 2, 256
    gen, order, inv, _ = routing(tokens, topk, 4, 0.1, 7)
    row = torch.randn((1, n), generator=gen, device=DEV).to(torch.bfloat16)
    y = torch.randn((tokens * topk, 2 * n), generator=gen, device=DEV).to(torch.bfloat16)[:, ::2]
    w = torch.randn((topk, tokens), generator=gen, device=DEV).t()
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream(DEV))
    dy, dw = gg.moe_unpermute_grad(row.expand(tokens, n), y, order, inv, w, stream=s)
    dx = gg.moe_permute_grad(y, inv, topk, stream=s)
    torch.cuda.current_stream(DEV).wait_stream(s)
    dy0, dw0 = gg.moe_unpermute_grad(row.repeat(tokens, 1), y.contiguous(), order, inv, w.contiguous())
    assert torch.equal(dy, dy0) and torch.equal(dw, dw0)
    assert torch.equal(dx, gg.moe_permute_grad(y.contiguous(), inv, topk))


def test_routing_gradients_replay_in_a_graph_and_repeat_bit_for_bit():
    tokens, topk, n, experts = 65, 4, 520, 16
    gen, order, inv, _ = routing(tokens, topk, experts, 0.1, 8)
    dout = torch.randn((tokens, n), generator=gen, device=DEV).to(torch.bfloat16)
    y = torch.randn((tokens * topk, n), generator=gen, device=DEV).to(torch.bfloat16)
    logits = torch.randn((tokens, experts), generator=gen, device=DEV)
    ids, w = gg.router_topk(logits, topk, "softmax")

    def step():
        dy, dw = gg.moe_unpermute_grad(dout, y, order, inv, w)
        return dy, dw, gg.moe_permute_grad(dy, inv, topk), gg.router_topk_grad(logits, ids, w, dw, "softmax")

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(DEV).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        dout.copy_(torch.randn(dout.shape, generator=gen, device=DEV))
        graph.replay()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
    assert not torch.equal(outs[0], eager[0])
    gg.moe_unpermute_grad(dout[:0], y[:0], order[:0], inv[:0], w[:0])   # no tokens
    assert gg.moe_permute_grad(y[:0], inv[:0], topk).shape == (0, n)
