"""GPU parity of MXFP4 quantisation and of the MXFP4 forward with plain 64-bit forms.

Quantisation is exact: codes, scales and values must be equal. The forward multiplies exactly
representable values and sums K products in fp32, each addition off by at most 2^-23 of the sum of the
magnitudes (an addition may truncate), then rounds once to bf16 (2^-8): the tolerances below.
"""
import numpy as np
import pytest
import torch

import group_gemm_gb300 as gg
import rdot_inputs as ri
from tests import _mxfp4 as mx
from tests._metrics import COSINE_MIN, cosine_to_rounded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def same_values(got, ref):
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(got.double()), torch.nan_to_num(ref))
    assert torch.equal(torch.signbit(got) & ~torch.isnan(got), torch.signbit(ref) & ~torch.isnan(ref))


def hard_rows(rows, k, dtype, seed):
    """Normal values over many magnitudes, with ties, zeros, subnormals, infinities and NaN."""
    g = gen(seed)
    x = torch.randn((rows, k), generator=g, device=DEV)
    x = torch.ldexp(x, torch.randint(-145, 120, (rows, 1), generator=g, device=DEV))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -5.0, 7.75, 0.0, -0.0, 4.0, 3.0],
                        device=DEV).repeat(2)
    for i in range(0, rows, 5):
        x[i, :32] = ties * 2.0 ** (i % 60 - 30)
    x[1::7, -32:] = 0
    if rows > 3:
        x[3, 0], x[2, k // 2] = float("nan"), float("-inf")
        x[0, k - 1] = torch.finfo(torch.float32).max
    return x.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (7, 96), (129, 1408), (3, 7168), (1000, 64), (4097, 544)])
def test_quantize_rows_is_exact(rows, k, dtype):
    x = hard_rows(rows, k, dtype, rows + k)
    codes, scales, values = gg.quantize_mxfp4(x, values=True)
    rc, rs, rv = mx.quantize(x)
    assert torch.equal(scales, rs)
    assert torch.equal(codes, mx.pack(rc))
    same_values(values, rv)
    c2, s2 = gg.quantize_mxfp4(x)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g,k,n", [(1, 32, 8), (2, 64, 128), (3, 160, 136), (5, 416, 264), (2, 4096, 72), (8, 256, 1024),
                                   (1, 1024, 520)])
def test_quantize_weight_is_exact(g, k, n, dtype):
    x = hard_rows(g * n, k, dtype, g + k + n).view(g, n, k)
    w = x.transpose(1, 2).contiguous()
    codes = torch.full((g, n, k // 2), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((g, -(-n // 128), -(-k // 128), 512), 0xFF, dtype=torch.uint8, device=DEV)
    values = torch.full((g, k, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    gg.rdot_quantize_mxfp4_weight(w, codes, scales, values)
    rc, rs, rv = mx.quantize(x)
    assert torch.equal(codes, mx.pack(rc))
    assert torch.equal(scales, mx.tile_scales(rs))       # zeros past N and K among them
    same_values(values.transpose(1, 2).contiguous(), rv)
    c2, s2 = gg.quantize_mxfp4_weight(w)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_quantize_takes_strided_inputs():
    x = torch.randn((64, 256), generator=gen(1), device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(gg.quantize_mxfp4(x[:, ::2]), gg.quantize_mxfp4(x[:, ::2].contiguous())))
    w = torch.randn((2, 64, 96), generator=gen(2), device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(gg.quantize_mxfp4_weight(w.transpose(1, 2)),
                                                 gg.quantize_mxfp4_weight(w.transpose(1, 2).contiguous())))
    assert gg.quantize_mxfp4(x[:0])[0].shape == (0, 128)


# ------------------------------------------------------------------------------ the forward
VARIANTS = {"pair": gg.RDOT_FLAG_CTA_PAIR, "skinny": gg.RDOT_FLAG_SKINNY, "default": 0}


def operands(m, k, n, groups, seed, spread=4):
    """Random codes, and scales that vary on every axis."""
    g = gen(seed)
    xq = torch.randint(0, 256, (m, k // 2), generator=g, device=DEV).to(torch.uint8)
    xs = torch.randint(127 - spread, 128 + spread, (m, k // 32), generator=g, device=DEV).to(torch.uint8)
    wq = torch.randint(0, 256, (groups, n, k // 2), generator=g, device=DEV).to(torch.uint8)
    ws = torch.randint(120 - spread, 121 + spread, (groups, n, k // 32), generator=g, device=DEV).to(torch.uint8)
    return xq, xs, wq, ws


def reference(xq, xs, wq, ws, sizes):
    x, w = mx.decode(xq, xs), mx.decode(wq, ws)
    out = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    at = 0
    for i, r in enumerate(sizes):
        out[at:at + r] = x[at:at + r] @ w[i].t()
        mag[at:at + r] = x[at:at + r].abs() @ w[i].abs().t()
        at += r
    return out, mag


def run(xq, xs, wq, ws, sizes, variant):
    m, n, k = xq.shape[0], wq.shape[1], 2 * xq.shape[1]
    plan = gg.Plan(m, k, n, len(sizes), "forward_mxfp4", "e2m1", "bf16", flags=VARIANTS[variant])
    if variant != "default":
        assert (plan.info["tile_m"], plan.info["tile_n"]) == {"pair": (256, 256), "skinny": (64, 128)}[variant]
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    gg.rdot_forward_mxfp4(plan.handle, xq, xs, wq, mx.tile_scales(ws),
                          torch.tensor(sizes, dtype=torch.int32, device=DEV), out, plan.workspace)
    return out, gg.rdot_read_status(plan.handle, plan.workspace)


def check(out, ref, mag, k):
    err = (out.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + k * 2.0 ** -23 * mag
    assert torch.all(err <= tol), f"worst {float((err - tol).max()):.3g} over, {int((err > tol).sum())} of {err.numel()}"


CASES = [
    (1, 32, 8, [1]),                                   # one row, one block, eight columns
    (2, 64, 128, [0, 1, 0, 1]),
    (1, 4096, 1024, [0, 0, 1]),
    (5, 96, 136, [2, 0, 3]),                           # K = 96: a half MMA step; N = 136
    (16, 160, 264, [16]),
    (48, 288, 40, [17, 0, 31]),                        # a second stage of one half step
    (64, 512, 256, [64]),
    (65, 512, 384, [65]),                              # a second token tile of one row
    (200, 640, 520, [130, 0, 70]),
    (300, 128, 128, [300]),
    (420, 1056, 144, [130, 0, 77, 200, 5]),            # K = 1056: 33 scale bytes a row
    (512, 256, 256, [0, 256, 256, 0]),
    (1000, 768, 776, [0, 313, 1, 0, 257, 300, 129]),
    (700, 1152, 264, [100, 0, 300, 200]),              # rows past the sum; 36 scale bytes a row
    (40, 7168, 512, [7, 0, 0, 1, 30]),
    (260, 256, 136, [i % 9 if i % 3 else 0 for i in range(65)]),      # more groups than a warp has lanes
    (1500, 64, 72, [1 + i % 2 if i % 4 else 0 for i in range(1024)]),   # the most groups a plan takes
]


@pytest.mark.parametrize("variant", list(VARIANTS))
@pytest.mark.parametrize("m,k,n,sizes", CASES)
def test_forward_parity(m, k, n, sizes, variant):
    xq, xs, wq, ws = operands(m, k, n, len(sizes), m + k)
    total = sum(sizes)
    xs[total:] = 255                                   # NaN rows past the sum must never leak
    out, status = run(xq, xs, wq, ws, sizes, variant)
    ref, mag = reference(xq, torch.where(xs == 255, 0, xs), wq, ws, sizes)
    assert status == 0
    assert torch.all(out[total:] == 0)
    check(out[:total], ref[:total], mag[:total], k)
    assert cosine_to_rounded(out.float(), ref.cpu().numpy()) >= COSINE_MIN


@pytest.mark.parametrize("variant", ["pair", "skinny"])
@pytest.mark.parametrize("vary", [(), ("x",), ("w",)])
def test_forward_is_exact_on_small_integers(vary, variant):
    """With unit scales, or powers of two on one operand whose sums stay within 24 bits, every partial
    sum is a multiple of the smallest product below 2^24 of them: the result is the exact sum, rounded
    once to bf16, and a scale read for the wrong row, column or block shows."""
    m, k, n, sizes = 200, 512, 264, [70, 0, 130]
    xq, xs, wq, ws = operands(m, k, n, len(sizes), 3)
    g = gen(4)
    xs.fill_(127)
    ws.fill_(127)
    if "x" in vary:
        xs.copy_(torch.randint(127, 131, xs.shape, generator=g, device=DEV))
    if "w" in vary:
        ws.copy_(torch.randint(127, 131, ws.shape, generator=g, device=DEV))
    out, _ = run(xq, xs, wq, ws, sizes, variant)
    assert torch.equal(out, reference(xq, xs, wq, ws, sizes)[0].to(torch.bfloat16))


@pytest.mark.parametrize("variant", ["pair", "skinny"])
def test_nan_scales_reach_their_rows_and_columns_only(variant):
    m, k, n, sizes = 40, 512, 256, [15, 25]
    xq, xs, wq, ws = operands(m, k, n, len(sizes), 5)
    xs[4, 3] = 255
    ws[1, 77, 9] = 255
    out, _ = run(xq, xs, wq, ws, sizes, variant)
    nan = torch.zeros((m, n), dtype=torch.bool, device=DEV)
    nan[4] = True
    nan[15:, 77] = True
    assert torch.equal(torch.isnan(out), nan)


@pytest.mark.parametrize("variant", ["pair", "skinny"])
def test_group_sizes_are_clamped_and_reported(variant):
    m, k, n = 60, 256, 136
    xq, xs, wq, ws = operands(m, k, n, 3, 6)
    out, status = run(xq, xs, wq, ws, [-4, 50, 40], variant)
    ref, mag = reference(xq, xs, wq, ws, [0, 50, 10])
    assert status == gg.RDOT_STATUS_BIT_GROUP_SIZES
    check(out, ref, mag, k)


def test_scales_at_any_byte_offset():
    m, k, n, sizes = 50, 512, 128, [20, 30]
    xq, xs, wq, ws = operands(m, k, n, 2, 7)
    want, _ = run(xq, xs, wq, ws, sizes, "pair")
    for off in (1, 4, 8):
        buf = torch.full((xs.numel() + 16,), 255, dtype=torch.uint8, device=DEV)
        view = buf[off:off + xs.numel()].view(xs.shape)
        view.copy_(xs)
        for variant in ("pair", "skinny"):
            assert torch.equal(run(xq, view, wq, ws, sizes, variant)[0], want)


def test_quantised_product_of_real_values_and_default_kernels():
    """quantize -> product through the high-level calls, against the 64-bit product of the quantised
    values; a few rows a group take the swapped kernel, more the pairs."""
    for m, groups, tile in ((6, 4, (64, 128)), (90, 4, (64, 128)), (500, 4, (64, 128)), (900, 4, (256, 256))):
        k, n = 1024, 512
        g = gen(m)
        x = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
        w = (0.02 * torch.randn((groups, k, n), generator=g, device=DEV))
        sizes = ri.multinomial_group_sizes(m, groups, 1).tolist()
        xq, xs, xv = gg.quantize_mxfp4(x, values=True)
        wq, ws, wv = gg.quantize_mxfp4_weight(w, values=True)
        out = gg.ragged_dot_mxfp4(xq, xs, wq, ws, torch.tensor(sizes, device=DEV))
        info = gg.Plan(m, k, n, groups, "forward_mxfp4", "e2m1", "bf16").info
        assert (info["tile_m"], info["tile_n"]) == tile
        at = 0
        for i, r in enumerate(sizes):
            a, b = xv[at:at + r].double(), wv[i].double()
            check(out[at:at + r], a @ b, a.abs() @ b.abs(), k)
            at += r


def test_two_streams_at_once_and_graph_replay():
    m, k, n, groups = 300, 512, 384, 3
    cases = [operands(m, k, n, groups, s) for s in (8, 9)]
    gs = torch.tensor([100, 0, 200], dtype=torch.int32, device=DEV)
    args = [(c[0], c[1], c[2], mx.tile_scales(c[3]), gs) for c in cases]
    serial = [gg.ragged_dot_mxfp4(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    outs = [[], []]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream(DEV))
    for _ in range(6):
        for i, st in enumerate(streams):
            outs[i].append(gg.ragged_dot_mxfp4(*args[i], stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(o, serial[i]) for i in range(2) for o in outs[i])
    # a graph of quantise + product, replayed on new rows and new sizes
    x = torch.randn((m, k), generator=gen(10), device=DEV)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        gg.ragged_dot_mxfp4(*gg.quantize_mxfp4(x), *args[0][2:])
    torch.cuda.current_stream(DEV).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gg.ragged_dot_mxfp4(*gg.quantize_mxfp4(x), *args[0][2:])
    for seed, sizes in ((11, [0, 150, 150]), (12, [299, 1, 0])):
        x.copy_(torch.randn(x.shape, generator=gen(seed), device=DEV))
        gs.copy_(torch.tensor(sizes, dtype=torch.int32))
        graph.replay()
        assert torch.equal(out, gg.ragged_dot_mxfp4(*gg.quantize_mxfp4(x), *args[0][2:]))


@pytest.mark.parametrize("variant", ["pair", "skinny"])
def test_stopping_early_leaves_the_context_usable(variant):
    """The wait limit set short enough that the pipelines' waits run out with work in flight: each call
    returns (stopped, with the timeout bit, or complete), and afterwards the default limit gives the
    same output as before."""
    m, k, n, sizes = (2048, 1024, 1024, [700, 0, 900, 448]) if variant == "pair" else (48, 1024, 1024, [20, 0, 28, 0])
    xq, xs, wq, ws = operands(m, k, n, len(sizes), 13)
    plan = gg.Plan(m, k, n, len(sizes), "forward_mxfp4", "e2m1", "bf16", flags=VARIANTS[variant])
    gs, wt = torch.tensor(sizes, dtype=torch.int32, device=DEV), mx.tile_scales(ws)
    out = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    call = lambda: gg.rdot_forward_mxfp4(plan.handle, xq, xs, wq, wt, gs, out, plan.workspace)
    call()
    want = out.clone()
    assert plan.status() == 0
    for ns in (1, 1_000, 20_000):
        gg.rdot_set_wait_timeout(plan.handle, ns)
        for _ in range(3):
            call()
            torch.cuda.synchronize()
            assert plan.status() in (0, gg.RDOT_STATUS_BIT_TIMEOUT)
        plan.clear_status()
    gg.rdot_set_wait_timeout(plan.handle, 0)
    call()
    assert plan.status() == 0 and torch.equal(out, want)


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements: the last rows are written where they belong."""
    m, k, n = 70000, 32, 32768
    xq, xs, wq, ws = operands(m, k, n, 2, 14)
    sizes = [1, m - 1]
    out, status = run(xq, xs, wq, ws, sizes, "default")
    assert status == 0
    x, w = mx.decode(xq[-300:], xs[-300:]), mx.decode(wq[1], ws[1])
    check(out[-300:], x @ w.t(), x.abs() @ w.abs().t(), k)
