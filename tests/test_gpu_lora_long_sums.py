"""Long contractions of the low-rank adapters: the tensor cores cut the sums they accumulate, so the kernels add up
stretches of 512 terms at most there (1024 of codes) and join the stretches in rounded fp32 additions.

Tolerances: within a stretch a term is off by at most a whole step of the sum, 2 U of it with U = 2^-24, so n terms in
stretches of 512 by (2 * 512 + n / 512) U times the sum of their magnitudes, however long the contraction. The
tests of many rows and columns set a one before many terms of less than a step, which a single cut sum loses.
"""
import pytest
import torch

import group_gemm_gb300 as gg
from tests.test_gpu_lora import H, close, make, ragged, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U = 2.0 ** -24
STRETCH = 512


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


# one long group of few columns (its rows divided over a cluster), and as many items as fill the SMs (undivided)
@pytest.mark.parametrize("groups,rows,r", [(1, 1 << 20, 16), (1, 1 << 20, 40), (1, 1 << 20, 64), (1, 1 << 20, 128),
                                           (160, 1 << 16, 16), (160, 1 << 16, 128)])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("order", [False, True])
def test_weight_gradient_of_many_rows(groups, rows, r, codes, order):
    m, width = groups * rows, 64
    small = 2.0 ** -28
    t = torch.full((groups, rows, r), small, dtype=torch.bfloat16, device=DEV)
    t[:, 0] = 1
    t = t.view(m, r)
    z = torch.ones((m, width), dtype=torch.bfloat16, device=DEV)
    scales = None
    if codes:
        z, scales = gg.quantize_mxfp8(z)
    gs = torch.full((groups,), rows, dtype=torch.int32, device=DEV)
    at = torch.arange(m - 1, -1, -1, dtype=torch.int32, device=DEV) if order else None
    dw = gg.lora_grad_weight(t, z, gs, at, scales).double()
    ref = 1 + (rows - 1) * small
    stretch = 2 * STRETCH if codes else STRETCH
    assert (dw - ref).abs().max() <= ((2 * stretch + rows / stretch) * U + U) * ref


@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("r", [16, 128])
def test_nan_codes_in_groups_of_several_stretches(r, order):
    """A NaN code reaches the sums of its group's column alone, whether the group has one stretch of rows or more,
    with several items to a block."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    sizes = [0, 1500, 3, 513, 512, 1024, 0, 64, 2049, 700] * 5
    m, width, groups = sum(sizes), 1152, len(sizes)
    t = torch.randn((m, r), generator=gen, device=DEV).to(torch.bfloat16)
    codes, scales = gg.quantize_mxfp8(torch.randn((m, width), generator=gen, device=DEV))
    at = torch.randperm(m, generator=gen, device=DEV).int() if order else None
    rows = torch.arange(m, device=DEV) if at is None else at.long()
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    clean = gg.lora_grad_weight(t, codes, gs, at, scales)
    group = torch.repeat_interleave(torch.arange(groups, device=DEV), gs.long())
    hit = torch.randint(0, m, (300,), generator=gen, device=DEV)
    col = torch.randint(0, width, (300,), generator=gen, device=DEV)
    codes[rows[hit], col] = 0x7f
    want = torch.zeros((groups, width), dtype=torch.bool, device=DEV)
    want[group[hit], col] = True
    dw = gg.lora_grad_weight(t, codes, gs, at, scales)
    want = want.unsqueeze(1).expand_as(dw)
    assert torch.equal(torch.isnan(dw), want) and torch.equal(dw[~want], clean[~want])


@pytest.mark.parametrize("m,k,groups,order", [
    (800 * 16, 57344, 800, False),      # 16-row tiles, a block each: four warps divide the columns
    (800 * 16, 57344, 800, True),
    (152 * 128 - 500, 57344, 1, False),  # 128-row tiles, a block each
    (152 * 128 - 500, 57344, 1, True),
])
@pytest.mark.parametrize("call", ["lora_forward", "lora_grad_input"])
@pytest.mark.parametrize("r", [8, 32, 56, 128])
def test_first_product_of_many_columns(m, k, groups, order, call, r):
    """Each row sums to a number just above the middle of two bf16 neighbours, so t is the upper one; without the
    terms that a single sum cuts off it would be the lower."""
    small = 1.5 * 2.0 ** -24                  # three quarters of a step of sums from 1 to 2, in each 16 columns
    steps = k // 16
    margin = 7.2e-5
    ref = 1 + 2.0 ** -8 + margin
    assert margin > (2 * STRETCH + k / STRETCH / 4 + 16) * U * ref
    w = torch.zeros(k, dtype=torch.float64)
    w[16::16] = small
    rest = ref - (steps - 1) * small
    for i in range(4):                        # its value in bf16 terms
        w[i] = float(torch.tensor(rest).to(torch.bfloat16))
        rest -= float(w[i])
    assert abs(rest) < 2.0 ** -30
    w = w.to(torch.bfloat16).to(DEV)
    first = w.expand(groups, r, k).contiguous()
    second = torch.zeros((groups, r, 64), dtype=torch.bfloat16, device=DEV)
    x = torch.ones((m, k), dtype=torch.bfloat16, device=DEV)
    gs = torch.full((groups,), m // groups, dtype=torch.int32, device=DEV)
    at = torch.arange(m - 1, -1, -1, dtype=torch.int32, device=DEV) if order else None
    down, up = (first, second) if call == "lora_forward" else (second, first)
    _, t = getattr(gg, call)(x, down, up, gs, at)
    assert torch.all(t == 1 + 2.0 ** -7)


# several stretches in a block, in clusters of all sizes, with stages that do not fill the last stretch
@pytest.mark.parametrize("m,k,groups", [(1700, 14336, 1), (2600, 8200, 1), (3300, 12296, 1), (4100, 7240, 1), (5200, 14336, 1), (7000, 4168, 2),
                                        (9000, 2056, 3), (2000, 6408, 40), (700, 14344, 6)])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("order", [False, True])
def test_first_product_of_several_stretches(m, k, groups, r, order):
    d = make(m, k, 136, groups, r, ragged(m, groups, r, 70) if groups > 1 else [m - 70], order, k)
    out, t = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"])
    ref, ref_t, tol, tol_t = reference(d["x"], d["down"], d["up"], d["sizes"].tolist(), d["order"], d["scale"], d["base_n"])
    close(t, ref_t, tol_t)
    close(out, ref, tol)
    # and t to what the stretches leave: a rounding to bf16 of a value that is off by their sums' errors
    _, exact, _, _ = reference(d["x"].abs(), d["down"].abs(), d["up"], d["sizes"].tolist(), d["order"], d["scale"].abs(), None)
    close(t, ref_t, H * ref_t.abs() + (1 + H) * (2 * STRETCH + k / STRETCH + 32) * U * exact)
