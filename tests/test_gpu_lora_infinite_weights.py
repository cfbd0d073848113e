"""Infinities and NaNs among the second product's weights of an adapter that has rows: its rows are not finite in that
column (t enters the product as two terms, whose infinities may have two signs: an infinity or NaN), and nothing else
changes."""
import pytest
import torch

import group_gemm_gb300 as gg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


# 16-row tiles and 128-row tiles (from about 1500 rows on), widths with and without a ragged end
@pytest.mark.parametrize("m,k,n,r", [(90, 64, 72, 8), (90, 136, 4096, 24), (200, 72, 1000, 64), (300, 64, 136, 128),
                                     (6000, 64, 72, 8), (6000, 200, 1096, 24), (6000, 64, 136, 64), (6000, 72, 1000, 128),
                                     (30000, 64, 200, 16)])
@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("call", ["lora_forward", "lora_grad_input"])
@pytest.mark.parametrize("base", ["none", "apart", "in place"])
def test_infinite_weights(m, k, n, r, order, call, base):
    gen = torch.Generator(device=DEV).manual_seed(m + r)
    sizes = [m // 3, 0, m // 2, m // 10]
    x = torch.randn((m, k), generator=gen, device=DEV).to(torch.bfloat16)
    first = (torch.randn((4, r, k), generator=gen, device=DEV) * k ** -0.5).to(torch.bfloat16)
    second = (torch.randn((4, r, n), generator=gen, device=DEV) * 0.1).to(torch.bfloat16)
    at = torch.randperm(m, generator=gen, device=DEV).int() if order else None
    rows = torch.arange(m, device=DEV) if at is None else at.long()
    mine = rows[m // 3:m // 3 + m // 2]              # the rows of adapter 2, whose weights are hit
    # rows whose t is a small whole number (the second of its two terms is 0), one with t = 0
    x[mine[::3]] = 0
    x[mine[::3], 0] = 1
    x[mine[5]] = 0
    first[2, :, 0] = torch.where(torch.arange(r, device=DEV) % 2 == 0, 1.0, -2.0).to(torch.bfloat16)
    b = torch.randn((m, n), generator=gen, device=DEV).to(torch.bfloat16) if base != "none" else None
    if b is not None:
        b[mine[7], 9], b[mine[10], 9] = INF, -INF
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)

    def run(w):
        down, up = (first, w) if call == "lora_forward" else (w, first)
        copy = None if b is None else b.clone()
        extra = {} if base != "in place" else {"out" if call == "lora_forward" else "dx": copy}
        return getattr(gg, call)(x, down, up, gs, at, base=copy, **extra)

    clean, clean_t = run(second)
    hit = second.clone()
    hit[2, 3, 5], hit[2, 4, 9], hit[2, r - 1, n - 1] = INF, -INF, INF
    hit[2, 0, 17], hit[2, 2, 17] = INF, INF          # the same column twice: of one sign or not, as t's signs are
    hit[2, 6, 21] = NAN
    columns = torch.tensor([5, 9, 17, 21, n - 1], device=DEV)
    out, t = run(hit)
    assert torch.equal(t, clean_t)
    other = torch.ones_like(out, dtype=torch.bool)
    other[mine.unsqueeze(1), columns] = False
    same = (out == clean) | (torch.isnan(out) & torch.isnan(clean))
    assert torch.all(same[other])
    got = out[mine][:, columns]
    assert not torch.isfinite(got).any()
    assert torch.isnan(got[:, 3]).all()              # the NaN weight's column
