"""int64 group sizes that 32 bits do not hold count as what they are: past all rows, or negative (no rows)."""
import pytest
import torch

import group_gemm_gb300 as gg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


@pytest.mark.parametrize("wide,plain", [([2 ** 32 + 5, 7], [100, 0]), ([3, 2 ** 40, 9], [3, 97, 0]), ([2 ** 31], [100]),
                                        ([-2 ** 32 + 50, 20], [0, 20]), ([2 ** 62, 2 ** 62, 2 ** 62], [100, 0, 0])])
def test_sizes_past_32_bits(wide, plain):
    m, k, n, r, g = 100, 64, 72, 8, len(wide)
    gen = torch.Generator(device=DEV).manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=gen, device=DEV).to(torch.bfloat16)
    x, dy, down, up = rn(m, k), rn(m, n), rn(g, r, k), rn(g, r, n)
    sizes = [torch.tensor(v, dtype=torch.int64, device=DEV) for v in (wide, plain)]
    for call in (lambda s: gg.lora_forward(x, down, up, s), lambda s: gg.lora_grad_input(dy, down, up, s),
                 lambda s: (gg.lora_grad_weight(dy[:, :r], x, s),)):
        for got, want in zip(call(sizes[0]), call(sizes[1])):
            assert torch.equal(got, want)
