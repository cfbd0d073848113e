"""More of the adapters' gradients: widths of the bf16 weight gradient that are no multiple of 32, high ranks whose rows
a cluster divides, results and inputs of more than 2^31 elements, and each element of every gradient against the
64-bit formula's and against differences of the 64-bit forward, with bounds that a gradient off by 5 % fails.

Tolerances as in test_gpu_lora.py: a term of an fp32 sum is off by 2 U of the sum, a rounding to bf16 by H = 2^-8 of
the value (half of a step, 2^-7 of the numbers from 1 to 2), t in the second product by H^2."""
import pytest
import torch

import group_gemm_gb300 as gg
from tests import _mxfp8
from tests.test_gpu_lora import H, U, clamped, close, randn, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def check_weight(m, width, r, sizes, order, codes, out_dtype):
    gen = torch.Generator(device=DEV).manual_seed(m + width)
    t, z = randn(gen, (m, r)), randn(gen, (m, width), 3.0)
    rows = torch.randperm(m, generator=gen, device=DEV) if order else torch.arange(m, device=DEV)
    zq, zs, z64 = z, None, z.double()
    if codes:
        zq, zs = gg.quantize_mxfp8(z)
        z64 = _mxfp8.decode(zq, zs)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    guard = torch.full((len(sizes) * r * width + 64,), 7.0, dtype=out_dtype, device=DEV)     # 64 elements behind it
    dw = guard[:len(sizes) * r * width].view(len(sizes), r, width)
    gg.lora_grad_weight(t, zq, gs, rows.int() if order else None, zs, dw=dw)
    for g, (b, e) in enumerate(clamped(sizes, m)):
        tg, zg = t[b:e].double(), z64[rows[b:e]]
        ref = tg.t() @ zg
        close(dw[g], ref, 2 * (e - b) * U * (tg.abs().t() @ zg.abs()) + (H if out_dtype is torch.bfloat16 else U) * ref.abs())
    assert torch.all(guard[dw.numel():] == 7)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("width", [8, 24, 72, 120, 136, 1000])
@pytest.mark.parametrize("m,r,sizes", [
    (1, 8, [0, 1]), (100, 24, [37, 0, 63]), (700, 128, [300, 400]),      # a block each
    (3000, 16, [3000]), (3000, 64, [1400, 1600]), (9000, 104, [9000]),   # a cluster divides the rows
    (9000, 8, [30] * 300),                                               # several items to a block
])
def test_weight_gradient_of_any_width(m, r, sizes, width, order, out_dtype):
    check_weight(m, width, r, sizes, order, False, out_dtype)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("r", [72, 96, 128])
@pytest.mark.parametrize("m,width,sizes", [(9000, 160, [9000]), (9001, 128, [9001]), (6000, 1024, [2900, 3100]), (5000, 2080, [1, 4999]),
                                           (4000, 4736, [4000]), (7000, 320, [2000, 0, 5000])])
def test_high_ranks_in_clusters(m, width, sizes, r, order, codes, out_dtype):
    check_weight(m, width, r, sizes, order, codes, out_dtype)


def test_gradient_of_more_than_32_bits():
    """A result whose last group lies behind the 2^31st element and the 2^32nd byte."""
    g, r, width, m = 1024, 128, 16640, 5
    assert (g - 1) * r * width > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(1)
    t, z = randn(gen, (m, r)), randn(gen, (m, width))
    gs = torch.zeros(g, dtype=torch.int32, device=DEV)
    gs[0], gs[-1] = 2, 3
    for zq, zs, z64 in ((z, None, z.double()), (*gg.quantize_mxfp8(z), None)):
        z64 = _mxfp8.decode(zq, zs) if z64 is None else z64
        dw = torch.full((g, r, width), 7.0, dtype=torch.bfloat16, device=DEV)
        gg.lora_grad_weight(t, zq, gs, z_scale=zs, dw=dw)
        for i, part in ((0, slice(0, 2)), (g - 1, slice(2, 5))):
            tg, zg = t[part].double(), z64[part]
            close(dw[i], tg.t() @ zg, 6 * U * (tg.abs().t() @ zg.abs()) + H * (tg.t() @ zg).abs())
        assert not dw[1:-1].any()
        del dw


@pytest.mark.parametrize("m", [2100, 4200])     # 16-row tiles, 128-row tiles
def test_order_into_more_than_32_bits(m):
    """An order that reaches rows behind the 2^31st element of x, base and dx, and of codes."""
    k, r, n = 1 << 20, 8, 64
    gen = torch.Generator(device=DEV).manual_seed(2)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    x[-3:] = randn(gen, (3, k))
    down, up = randn(gen, (2, r, k), 2.0 ** -10), randn(gen, (2, r, n))
    order = torch.arange(m - 1, -1, -1, dtype=torch.int32, device=DEV)       # the last rows come first
    gs = torch.tensor([3, m - 3], dtype=torch.int32, device=DEV)
    out, t = gg.lora_forward(x, down, up, gs, order)
    ref, ref_t, tol, tol_t = reference(x[-3:], down[:1], up[:1], [3], torch.tensor([2, 1, 0], device=DEV), None, None)
    close(t[:3], ref_t, tol_t)
    close(out[-3:], ref, tol)
    assert not out[:-3].any() and not t[3:].any()
    tg, want = t[:3].double(), x[-3:].flip(0)
    mag = tg.abs().t() @ want.double().abs()
    dw = gg.lora_grad_weight(t, x, gs, order)
    close(dw[0], tg.t() @ want.double(), 6 * U * mag + U * mag)
    assert not dw[1].any()
    del dw
    codes, scales = torch.zeros((m, k), dtype=torch.uint8, device=DEV), torch.full((m, k // 32), 127, dtype=torch.uint8, device=DEV)
    codes[-3:], scales[-3:] = gg.quantize_mxfp8(x[-3:])
    z64 = _mxfp8.decode(codes[-3:], scales[-3:]).flip(0)
    dw = gg.lora_grad_weight(t, codes, gs, order, scales)
    close(dw[0], tg.t() @ z64, 7 * U * (tg.abs().t() @ z64.abs()))
    assert not dw[1].any()
    del dw, codes, scales
    dy = torch.zeros((m, n), dtype=torch.bfloat16, device=DEV)
    dy[-3:] = out[-3:]
    dx, dt = gg.lora_grad_input(dy, down, up, gs, order, base=x, dx=None)
    ref, ref_t, tol, tol_t = reference(dy[-3:], up[:1], down[:1], [3], torch.tensor([2, 1, 0], device=DEV), None, x[-3:])
    close(dt[:3], ref_t, tol_t)
    close(dx[-3:], ref, tol)
    assert not dx[:-3].any()


def violations(got, ref, tol):
    return int((~((got.double() - ref).abs() <= tol)).sum())


@pytest.mark.parametrize("many", [False, True])     # 16-row tiles, 128-row tiles
@pytest.mark.parametrize("r", [8, 24])
def test_each_element_of_the_gradients(many, r):
    k, n, g = 24, 40, 3
    sizes = [1700, 0, 2300] if many else [5, 0, 9]
    m = sum(sizes) + 4
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, dy, down, up = randn(gen, (m, k)), randn(gen, (m, n)), randn(gen, (g, r, k), 0.3), randn(gen, (g, r, n), 0.3)
    order = torch.randperm(m, generator=gen, device=DEV).int()
    scale = torch.rand(g, generator=gen, device=DEV) + 0.5
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    group = torch.cat([torch.full((s,), i, device=DEV) for i, s in enumerate(sizes)] + [torch.full((4,), -1, device=DEV)])
    of_row = torch.empty(m, dtype=torch.long, device=DEV)
    of_row[order.long()] = group
    live = (of_row >= 0).double().unsqueeze(1)
    at = of_row.clamp(min=0)

    def loss(x, down, up):                          # x [.., m, k], down [.., g, r, k], up [.., g, r, n]
        t = torch.einsum("...mk,...mrk->...mr", x, down[..., at, :, :]) * scale.double()[at].unsqueeze(1) * live
        return (torch.einsum("...mr,...mrn->...mn", t, up[..., at, :, :]) * dy.double()).sum((-1, -2))

    _, t = gg.lora_forward(x, down, up, gs, order, scale)
    dx, dt = gg.lora_grad_input(dy, down, up, gs, order, scale)
    got = (dx, gg.lora_grad_weight(dt, x, gs, order), gg.lora_grad_weight(t, dy, gs, order))

    leaves = [v.double().requires_grad_() for v in (x, down, up)]
    grads = torch.autograd.grad(loss(*leaves), leaves)
    x64, down64, up64 = (v.detach() for v in leaves)
    # the loss is linear in each input: its differences along single elements are the gradient's, with the rounding
    # of the two losses in 64 bits over the step
    for which, ref in enumerate(grads):
        flat = ref.flatten()
        pick = torch.randint(0, flat.numel(), (20,), generator=gen, device=DEV)
        for i in pick.tolist():
            hi, lo = [x64, down64, up64], [x64, down64, up64]
            step = torch.zeros_like(flat)
            step[i] = 1
            hi[which] = hi[which] + step.view(ref.shape)
            lo[which] = lo[which] - step.view(ref.shape)
            diff = float(loss(*hi) - loss(*lo)) / 2
            assert abs(diff - float(flat[i])) <= 1e-9 * (1 + abs(diff)) * m
    # t, dt and dx against the formula's, element by element; the adapters' gradients against the formula's of the t and dt
    # that they were given, which differ from the exact ones by those roundings
    s = scale.double()[at].unsqueeze(1) * live
    t64 = torch.einsum("mk,mrk->mr", x64, down64[at]) * s
    tm = torch.einsum("mk,mrk->mr", x64.abs(), down64[at].abs()) * s
    dt64 = torch.einsum("mn,mrn->mr", dy.double(), up64[at]) * s
    dtm = torch.einsum("mn,mrn->mr", dy.double().abs(), up64[at].abs()) * s
    err_t, err_dt = 2 * (k + 2) * U * tm, 2 * (n + 2) * U * dtm           # of t and dt before they are rounded
    member = torch.nn.functional.one_hot(at, g).double() * live
    unsorted = lambda v: torch.empty_like(v).index_copy_(0, order.long(), v)
    sums = lambda a, b: torch.einsum("mg,mr,mk->grk", member, a, b.double())
    t_rows, dt_rows = unsorted(t).double(), unsorted(dt).double()
    checks = {"t": (unsorted(t), t64, err_t + H * (t64.abs() + err_t)),
              "dt": (unsorted(dt), dt64, err_dt + H * (dt64.abs() + err_dt)),
              "dx": (dx, grads[0], torch.einsum("mr,mrk->mk", err_dt + H * H * dt64.abs() + 2 * (2 * r + 2) * U * dtm, down64[at].abs())
                     + H * grads[0].abs()),
              "ddown": (got[1], sums(dt_rows, x), 2 * max(sizes) * U * sums(dt_rows.abs(), x.abs())),
              "dup": (got[2], sums(t_rows, dy), 2 * max(sizes) * U * sums(t_rows.abs(), dy.abs()))}
    for name, (v, ref, tol) in checks.items():
        assert violations(v, ref, tol) == 0, name
        # what the bounds tell apart: most elements that a few percent move at all
        for wrong in (1.05, 0.95, -1.0):
            assert violations(wrong * v.double(), ref, tol) > 0.8 * int((ref != 0).sum()), (name, wrong)
    # and the whole of it: the gradient of the exact formula, off by the roundings of t and dt
    assert violations(got[1], grads[1], checks["ddown"][2] + sums(checks["dt"][2], x.abs())) == 0
    assert violations(got[2], grads[2], checks["dup"][2] + sums(checks["t"][2], dy.abs())) == 0
