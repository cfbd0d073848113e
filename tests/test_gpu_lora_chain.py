"""Long chains of the adapter calls on one stream, the many-row form behind itself, the weight gradient and the library's
products: kernels that begin while the one before still runs share the SMs' tensor memory with it, on one stream or two.
Every result equals the same call's alone."""
import pytest
import torch

import group_gemm_gb300 as gg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def case(m, k, n, g, r, order, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s, std=1.0: (torch.randn(s, generator=gen, device=DEV) * std).to(torch.bfloat16)
    gs = torch.full((g,), m // g, dtype=torch.int32, device=DEV)
    at = torch.randperm(m, generator=gen, device=DEV).int() if order else None
    x, dy, down, up, w = rn(m, k), rn(m, n), rn(g, r, k, std=k ** -0.5), rn(g, r, n, std=0.1), rn(g, k, n, std=k ** -0.5)
    zq, zs = gg.quantize_mxfp8(x)

    def step(stream=None):
        base = gg.ragged_dot(x, w, gs, stream=stream)
        y, t = gg.lora_forward(x, down, up, gs, at, base=base, stream=stream)
        y2, _ = gg.lora_forward(x, down, up, gs, at, base=y, stream=stream)
        dup = gg.lora_grad_weight(t, dy, gs, at, stream=stream)
        dx, dt = gg.lora_grad_input(dy, down, up, gs, at, stream=stream)
        ddown = gg.lora_grad_weight(dt, zq, gs, at, zs, stream=stream)
        dw = gg.grad_weight(x, y2, gs, stream=stream)
        return y2, dup, dx, ddown, dw

    return step


# ranks that take 128 to 512 columns of tensor memory, sizes that take the 128-row form with a block or two an SM
CASES = [(8192, 512, 1024, 8, 16, False), (6000, 256, 512, 4, 64, True), (4096, 1024, 256, 2, 128, False), (12000, 128, 128, 40, 32, True)]


def together(steps, streams, times):
    refs = [step() for step in steps]
    for ref in refs:
        assert all(torch.isfinite(v).all() for v in ref)
    torch.cuda.synchronize()
    outs = []
    for _ in range(times):
        outs.append([step(s) for step, s in zip(steps, streams)])
    torch.cuda.synchronize()
    for round_ in outs:
        for ref, got in zip(refs, round_):
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert gg.rdot_lora_read_status() == 0


def test_one_stream():
    together([case(*c, i) for i, c in enumerate(CASES)], [None] * len(CASES), 25)


def test_two_streams():
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    together([case(*c, i) for i, c in enumerate(CASES)], [streams[i % 2] for i in range(len(CASES))], 25)


def test_captured():
    steps = [case(*c, i) for i, c in enumerate(CASES)]
    refs = [step() for step in steps]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [[step() for step in steps] for _ in range(4)]
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for round_ in outs:
        for ref, got in zip(refs, round_):
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
