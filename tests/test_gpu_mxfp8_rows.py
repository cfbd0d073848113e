"""GPU parity of the MXFP8 quantiser of rows and of its inverse with a plain 64-bit form: codes and scales are
exact, and so are the restored values in fp32; in bf16 they are rounded to nearest even below 2^-126."""
import pytest
import torch

import group_gemm_gb300 as gg
from tests import _mxfp8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def check(x):
    codes, scales = gg.quantize_mxfp8(x)
    ref_c, ref_s, values = _mxfp8.quantize(x)
    assert torch.equal(codes, ref_c) and torch.equal(scales, ref_s)
    for dtype in (torch.float32, torch.bfloat16):
        got = gg.dequantize_mxfp8(codes, scales, dtype)
        ref = values.to(torch.float32).to(dtype)     # fp32 holds every value: one rounding
        assert got.dtype == dtype and torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 7168), (3, 96), (61, 1408), (257, 32), (129, 4096), (5000, 2080)])
def test_round_trip(rows, k, dtype):
    gen = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn((rows, k), generator=gen, device=DEV)
    x *= torch.exp2(torch.randint(-140, 120, (rows, k // 32), generator=gen, device=DEV).float()).repeat_interleave(32, 1)
    check(x.to(dtype))


def test_many_rows():
    gen = torch.Generator(device=DEV).manual_seed(0)
    check(torch.randn((9000, 4096), generator=gen, device=DEV).to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_special_values(dtype):
    """Blocks of zeros, of -0, with an infinity or a NaN, of subnormals, at the border of a scale (amax 448 x 2^e
    and the next number), and of halfway elements."""
    x = torch.zeros((16, 64), device=DEV)
    x[0] = -0.0
    x[1, 5], x[2, 5], x[3, 40] = float("inf"), float("-inf"), float("nan")
    x[1, 33] = 7.0
    x[4] = torch.arange(64, device=DEV) * 2.0 ** -149
    x[5], x[6] = 3.3e38, -2.0 ** -126
    for i, e in enumerate((-120, -119, -8, 0, 100)):
        eps = 2.0 ** -7 if dtype is torch.bfloat16 else 2.0 ** -23
        x[7 + i, 0] = 448 * 2.0 ** e
        x[7 + i, 32] = 448 * 2.0 ** e * (1 + eps)
        x[7 + i, 1:32] = torch.arange(31, device=DEV) * 2.0 ** (e - 10)   # halves of the smallest step
        x[7 + i, 33:] = 448 * 2.0 ** e * torch.linspace(-1, 1, 31, device=DEV)
    x[12] = torch.linspace(-1, 1, 64, device=DEV)
    check(x.to(dtype))


def test_every_code_and_scale():
    """Restoring takes any code and scale, the quantiser's or not: NaN for codes 127 and 255 and for scale 255."""
    codes = torch.arange(256, device=DEV, dtype=torch.uint8).repeat(32, 1)        # 8 blocks a row
    scales = torch.arange(256, device=DEV, dtype=torch.uint8).view(32, 8)
    ref = _mxfp8.decode(codes, scales)
    for dtype in (torch.float32, torch.bfloat16):
        got, r = gg.dequantize_mxfp8(codes, scales, dtype), ref.to(torch.float32).to(dtype)
        assert torch.equal(torch.isnan(got), torch.isnan(r))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(r))


def test_feeds_the_mxfp8_forward():
    """Codes and scales are the forward's lhs as they are."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    m, k, n, g = 300, 256, 128, 3
    x = torch.randn((m, k), generator=gen, device=DEV).to(torch.bfloat16)
    w = torch.randn((g, k, n), generator=gen, device=DEV)
    gs = torch.tensor([100, 0, 150], dtype=torch.int32, device=DEV)
    xq, xs = gg.quantize_mxfp8(x)
    wq, ws, wv = _mxfp8.quantize(w.transpose(1, 2).contiguous())     # blocks along K
    out = gg.ragged_dot_mxfp8(xq, xs, wq.transpose(1, 2).contiguous(), ws.transpose(1, 2).contiguous(), gs)
    xv = _mxfp8.decode(xq, xs)
    ref = torch.zeros((m, n), dtype=torch.float64, device=DEV)
    ref[:100] = xv[:100] @ wv[0].t()
    ref[100:250] = xv[100:250] @ wv[2].t()
    mag = xv.abs().sum(1, keepdim=True) * wv.abs().amax()
    err = (out.double() - ref).abs()
    assert torch.all(err <= 2.0 ** -8 * ref.abs() + k * 2.0 ** -23 * mag)


def test_streams_graph_and_strides():
    gen = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn((64, 300), generator=gen, device=DEV)[:, 6:262]                # rows of a wider tensor
    codes, scales = gg.quantize_mxfp8(x)
    assert torch.equal(codes, _mxfp8.quantize(x)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c2, s2 = gg.quantize_mxfp8(x, stream=side)
    back = gg.dequantize_mxfp8(c2, s2, stream=side)
    side.synchronize()
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    xg = x.contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cg, sg = gg.quantize_mxfp8(xg)
        vg = gg.dequantize_mxfp8(cg, sg)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(vg, back)
    xg.copy_(-x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(vg, -back)
