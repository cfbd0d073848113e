"""The MXFP4 forward's persistent loops across tiles of several K stages, against the 64-bit product.

The shapes follow from the device's number of SMs, so that the loops are certain to run: on the pair
kernel three tiles and more a pair (a tile that starts in the middle of the rings, accumulators that
overlap, the row-scale buffers flipping after a partial group of stages); on the swapped kernel two whole
items a CTA and a rest that is cut into quarters, halves or not at all, with N ending inside an item.
"""
import pytest
import torch

import group_gemm_gb300 as gg
from tests._metrics import COSINE_MIN, cosine_to_rounded
from tests.test_gpu_mxfp4 import check, operands, reference, run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
# stages of 256 elements: 5, the last of 160; 9, full; 10, the last of 32 elements (73 scale bytes a row);
# 11 (88 scale bytes); 17 (136)
WIDTHS = [1184, 2304, 2336, 2816, 4352]


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def sm_count():
    return torch.cuda.get_device_properties(DEV).multi_processor_count


def parity(m, k, n, sizes, variant, seed):
    xq, xs, wq, ws = operands(m, k, n, len(sizes), seed)
    total = sum(sizes)
    xs[total:] = 255
    out, status = run(xq, xs, wq, ws, sizes, variant)
    ref, mag = reference(xq, torch.where(xs == 255, 0, xs), wq, ws, sizes)
    assert status == 0 and torch.all(out[total:] == 0)
    check(out[:total], ref[:total], mag[:total], k)
    assert cosine_to_rounded(out.float(), ref.cpu().numpy()) >= COSINE_MIN


@pytest.mark.parametrize("k", WIDTHS)
def test_pair_kernel_over_several_tiles(k):
    sizes = [700, 1, 0, 513, 300, 256]
    row_tiles = sum(-(-s // 256) for s in sizes)
    pairs = sm_count() // 2
    column_tiles = -(-7 * pairs // (2 * row_tiles))              # 3.5 tiles a pair
    n = 256 * column_tiles - 120
    info = gg.Plan(1800, k, n, len(sizes), "forward_mxfp4", "e2m1", "bf16", flags=gg.RDOT_FLAG_CTA_PAIR).info
    assert row_tiles * column_tiles > 3 * (info["grid_ctas"] // 2)
    parity(1800, k, n, sizes, "pair", k)


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("width,rest", [(1, 0.15), (2, 0.4), (4, 0.75)])
@pytest.mark.parametrize("last", [40, 72, 128])                   # columns of the last 128-column item
def test_swapped_kernel_over_whole_items_and_a_cut_rest(width, rest, last, k):
    sizes = [40, 0, 70]                                           # one token tile and two
    sms = sm_count()
    atoms = round((2 + rest) * sms / 3)
    left = 3 * atoms - 2 * sms
    assert 0 < left < sms and width == (1 if 4 * left <= sms else 2 if 2 * left <= sms else 4)
    n = 128 * (atoms - 1) + last
    info = gg.Plan(115, k, n, len(sizes), "forward_mxfp4", "e2m1", "bf16", flags=gg.RDOT_FLAG_SKINNY).info
    assert info["grid_ctas"] == sms
    parity(115, k, n, sizes, "skinny", k + last)
