"""GPU parity of the low-rank adapters (grouping, forward, gradient of the input, gradients of the adapters)
with plain 64-bit forms of the same formulas on the same inputs.

Tolerances follow from the arithmetic. A term added to an fp32 sum on the tensor cores is off by at most a
whole step of the sum, 2 U with U = 2^-24 (they may cut instead of rounding), so n terms by 2 n U times the
sum of their magnitudes; a rounding to bf16 is off by at most H = 2^-8 of the value. t enters the second
product as hi + lo: lo is rounded, |lo| <= H |t|, so t is off by H^2 |t|.
"""
import pytest
import torch

import group_gemm_gb300 as gg
from tests import _mxfp8

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U, H = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _built():
    gg.build()
    gg.load()


def close(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol + TINY)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float((err - tol).max()):.3g} over"


def randn(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(torch.bfloat16)


def clamped(sizes, m):
    """[(start, end)] of each group under the reading of negative and too large sizes."""
    at, out = 0, []
    for s in sizes:
        b, at = min(at, m), at + max(s, 0)
        out.append((b, min(at, m)))
    return out


def reference(x, first, second, sizes, order, scale, base):
    """(out, t, tolerance of out, tolerance of t) in 64 bits."""
    m, width = x.shape[0], second.shape[2]
    rows = torch.arange(m, device=DEV) if order is None else order.long()
    out = torch.zeros((m, width), dtype=torch.float64, device=DEV) if base is None else base.double()
    t = torch.zeros((m, first.shape[1]), dtype=torch.float64, device=DEV)
    tol, tol_t = torch.zeros_like(out), torch.zeros_like(t)
    k, r = x.shape[1], first.shape[1]
    for g, (b, e) in enumerate(clamped(sizes, m)):
        if b == e:
            continue
        i, s = rows[b:e], 1.0 if scale is None else float(scale[g])
        xg, f, w = x[i].double(), first[g].double(), second[g].double()
        t[b:e] = s * (xg @ f.t())
        mag = abs(s) * (xg.abs() @ f.abs().t())
        tol_t[b:e] = (2 * k + 2) * U * mag                          # K terms, the scale's product
        prod = t[b:e].abs() @ w.abs()
        out[i] += t[b:e] @ w
        tol[i] = (tol_t[b:e] + H * H * t[b:e].abs()) @ w.abs() + 2 * (2 * r + 2) * U * (prod + (0 if base is None else base[i].double().abs()))
    return out, t, tol + H * out.abs() * (1 if base is None else 1), tol_t + H * t.abs()


def ragged(m, g, seed, spare=0):
    """g group sizes that sum to m - spare: an empty one, short and long ones."""
    cuts = torch.randint(0, m - spare + 1, (g - 1,), generator=torch.Generator().manual_seed(seed)).sort().values.tolist()
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [m - spare])]
    if g > 2:
        sizes[1], sizes[2] = 0, sizes[1] + sizes[2]
    return sizes


def make(m, k, n, g, r, sizes, order, seed=0, base=True, scale=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    d = {"x": randn(gen, (m, k)), "dy": randn(gen, (m, n)), "down": randn(gen, (g, r, k), k ** -0.5), "up": randn(gen, (g, r, n), 0.1)}
    d["sizes"] = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    d["order"] = torch.randperm(m, generator=gen, device=DEV).int() if order else None
    d["scale"] = torch.randn(g, generator=gen, device=DEV) if scale else None
    d["base_n"] = randn(gen, (m, n)) if base else None
    d["base_k"] = randn(gen, (m, k)) if base else None
    return d


APPLY = [       # m, k, n, r, group sizes, order, base, scale
    (1, 64, 64, 8, [1], False, True, True), (1, 4096, 4096, 16, [0, 0, 1, 0], True, True, True),
    (1, 8, 8, 8, [0], False, True, False), (5, 264, 72, 8, [1, 0, 3], True, False, True),
    (16, 128, 128, 16, [16], False, True, False), (17, 136, 1000, 24, [16, 1], True, True, True),
    (64, 4096, 1408, 16, [1] * 50 + [0] * 200 + [2] * 6, True, True, True),
    (64, 1000, 2048, 128, [30, 2, 0, 9], True, True, True), (63, 72, 8, 64, [0, 5, 50], False, False, False),
    (64, 128, 256, 16, [64], False, True, True), (65, 128, 256, 32, [65], True, True, True),
    (200, 520, 264, 40, [3, 0, 129, 64], True, True, True), (700, 1408, 2048, 64, [333, 0, 1, 300], False, True, True),
    (515, 2048, 520, 96, [200, 100, 0, 215], True, True, False), (515, 200, 1032, 128, [515], False, True, True),
    (2061, 7168, 264, 64, [400, 0, 1600], True, True, True), (3000, 512, 4096, 16, [1000, 900, 64, 65, 63, 500], False, True, True),
    (300, 64, 64, 16, [0, 0], True, True, True), (300, 64, 64, 16, [0, 0], False, False, True),
    (128, 256, 192, 8, [-5, 60, 1 << 30, 7], True, True, True), (40, 64, 192, 16, [0] * 1023 + [33], True, True, True),
    (5000, 136, 136, 8, [5] * 1000, False, True, True),
]


# Many rows: the 128-row form, with clusters of 4, 2 and 1 and a deep ring, of 2 and 1 and a short one
for _i, (_m, _g) in enumerate([(4100, 1), (4100, 3), (8000, 3), (12000, 40), (7000, 60), (20000, 9), (70000, 2)]):
    for _r in ((8, 24, 40, 128) if _m < 20000 else (16, 64)):
        APPLY.append((_m, 200 + 64 * _i, 328 - 8 * _i, _r, ragged(_m, _g, _i, 130), _r % 16 == 0, _i % 3 != 1, _r != 24))
APPLY += [(4500, 8, 8, 8, [4500], True, True, True), (4500, 2056, 8, 16, [4000, 100], False, True, True),
          (4500, 64, 2056, 32, [100, 129, 4200], True, False, True), (4500, 64, 64, 64, [0, 0], True, False, False),
          (4500, 64, 64, 64, [0, 0], True, True, False), (5000, 72, 136, 16, [-3, 2000, 1 << 30, 5], True, True, True)]
# Few tiles, whose columns several clusters divide; 16-row tiles beside the border to the 128-row form at each size of rank
APPLY += [(1, 4096, 14336, 32, [0, 1, 0], True, True, True), (2, 264, 8200, 64, [1], False, True, True),
          (9, 4096, 14336, 16, [1, 0, 3, 1, 1], True, True, True), (20, 520, 5000, 128, [7, 1, 9], True, False, True)]
for _i, (_m, _g) in enumerate([(90, 80), (128, 128), (520, 16), (768, 24), (800, 40), (1200, 32), (2000, 32), (3000, 32), (3000, 4)]):
    for _r in (16, 32, 56, 104):
        APPLY.append((_m, 328 - 8 * _i, 200 + 64 * _i, _r, ragged(_m, _g, 50 + _i, 9), _i % 4 != 1, _i % 3 != 2, _r != 32))
# Clusters of 7, 6, 5 and 3 blocks, which do not divide a tile's rows
for _i, _m in enumerate([4000, 4700, 5500, 3000]):
    for _r in (16, 32, 64, 72):
        APPLY.append((_m, 1032 + 8 * _i, 960, _r, ragged(_m, 12 if _i < 3 else 60, 70 + _i, 40), _r != 32 or _i == 3, True, True))


@pytest.mark.parametrize("m,k,n,r,sizes,order,base,scale", APPLY)
def test_forward(m, k, n, r, sizes, order, base, scale):
    d = make(m, k, n, len(sizes), r, sizes, order, 1, base, scale)
    out, t = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"])
    ref, ref_t, tol, tol_t = reference(d["x"], d["down"], d["up"], sizes, d["order"], d["scale"], d["base_n"])
    close(t, ref_t, tol_t)
    close(out, ref, tol)


@pytest.mark.parametrize("m,k,n,r,sizes,order,base,scale", APPLY)
def test_grad_input(m, k, n, r, sizes, order, base, scale):
    d = make(m, k, n, len(sizes), r, sizes, order, 2, base, scale)
    dx, dt = gg.lora_grad_input(d["dy"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_k"])
    ref, ref_t, tol, tol_t = reference(d["dy"], d["up"], d["down"], sizes, d["order"], d["scale"], d["base_k"])
    close(dt, ref_t, tol_t)
    close(dx, ref, tol)


WEIGHT = [      # m, width, r, group sizes, order
    (1, 32, 8, [1], False), (1, 4096, 16, [0, 1, 0], True), (3, 96, 8, [0, 3], True), (64, 160, 16, [64], False),
    (65, 128, 32, [65], True), (17, 4128, 24, [16, 0, 1], True), (200, 1408, 64, [63, 1, 0, 130], True),
    (515, 2048, 40, [100, 415], False), (700, 1056, 128, [333, 0, 300], True), (4099, 512, 64, [4000, 64, 30], True),
    (300, 64, 16, [0, 0], True), (128, 64, 8, [-5, 60, 1 << 30, 7], False), (2000, 224, 96, [1] * 1000 + [1000], True),
    (9000, 128, 16, [9000], False),
    (3000, 2048, 16, [2990], True), (3000, 4736, 8, [3000], False), (2600, 3200, 40, [2600], True),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("m,width,r,sizes,order", WEIGHT)
def test_grad_weight(m, width, r, sizes, order, codes, out_dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    t, z = randn(gen, (m, r)), randn(gen, (m, width), 3.0)
    rows = torch.randperm(m, generator=gen, device=DEV) if order else torch.arange(m, device=DEV)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    bounds = clamped(sizes, m)
    past = bounds[-1][1]
    t[past:] = float("nan")                 # rows of no group are never read into the result
    z[rows[past:]] = float("nan")
    zq, zs, z64 = z, None, z.double()
    if codes:
        zq, zs = gg.quantize_mxfp8(z)
        z64 = _mxfp8.decode(zq, zs)
    dw = gg.lora_grad_weight(t, zq, gs, rows.int() if order else None, zs, out_dtype)
    assert dw.dtype == out_dtype and dw.shape == (len(sizes), r, width)
    for g, (b, e) in enumerate(bounds):
        tg, zg = t[b:e].double(), z64[rows[b:e]]
        ref = tg.t() @ zg
        tol = 2 * (e - b) * U * (tg.abs().t() @ zg.abs())
        close(dw[g], ref, tol + (H if out_dtype is torch.bfloat16 else U) * ref.abs())
        if b == e:
            assert torch.all(dw[g] == 0)


def test_grad_weight_without_rows():
    dw = torch.full((3, 8, 64), float("nan"), device=DEV)
    empty = torch.empty((0, 8), dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([4, 0, 1], dtype=torch.int32, device=DEV)
    gg.lora_grad_weight(empty, torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), gs, dw=dw)
    assert torch.all(dw == 0)
    out, t = gg.lora_forward(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), *(
        torch.zeros((3, 8, w), dtype=torch.bfloat16, device=DEV) for w in (64, 32)), gs)
    assert out.shape == (0, 32) and t.shape == (0, 8)


def test_grad_weight_codes_of_any_kind():
    """Scales from the smallest to the largest finite, subnormal codes, and a NaN code or scale, which reaches the
    sums of its own columns alone."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    m, width, r = 100, 96, 16
    codes = torch.randint(0, 127, (m, width), generator=gen, device=DEV, dtype=torch.uint8)
    codes += 128 * torch.randint(0, 2, (m, width), generator=gen, device=DEV, dtype=torch.uint8)
    gs = torch.tensor([m], dtype=torch.int32, device=DEV)
    for s in (9, 10, 60, 127, 140, 240):           # 2^-118: the smallest code, 2^-9 of it, is a bf16 number still
        scales = torch.full((m, 3), s, dtype=torch.uint8, device=DEV)
        t = randn(gen, (m, r), 2.0 ** (100 - s) if s > 200 else 1.0)
        z = _mxfp8.decode(codes, scales)
        ref, mag = t.double().t() @ z, t.double().abs().t() @ z.abs()
        dw = gg.lora_grad_weight(t, codes, gs, z_scale=scales)[0]
        close(dw, ref, 2 * m * U * mag + U * ref.abs())
    scales = torch.full((m, 3), 127, dtype=torch.uint8, device=DEV)
    t = randn(gen, (m, r))
    codes[7, 40] = 0xff
    scales[50, 0] = 255
    dw = gg.lora_grad_weight(t, codes, gs, z_scale=scales)[0]
    assert torch.isnan(dw[:, :32]).all() and torch.isnan(dw[:, 40]).all()
    dw[:, 40] = 0
    assert torch.isfinite(dw[:, 32:]).all()


def test_scales_of_any_alignment():
    """A checkpoint's scales may start at any byte, with rows of any number of them."""
    gen = torch.Generator(device=DEV).manual_seed(20)
    m, width, r = 150, 160, 8
    t, z = randn(gen, (m, r)), randn(gen, (m, width))
    codes, scales = gg.quantize_mxfp8(z)
    gs = torch.tensor([100, 30], dtype=torch.int32, device=DEV)
    ref = gg.lora_grad_weight(t, codes, gs, z_scale=scales)
    buf = torch.empty(scales.numel() + 3, dtype=torch.uint8, device=DEV)
    for shift in (1, 2, 3):
        odd = buf[shift:shift + scales.numel()].view(scales.shape)
        odd.copy_(scales)
        assert torch.equal(gg.lora_grad_weight(t, codes, gs, z_scale=odd), ref)


@pytest.mark.parametrize("m,g", [(1, 1), (31, 4), (32, 1), (33, 1024), (64, 256), (1000, 7), (4096, 64), (4097, 1023),
                                 (16384, 64), (16385, 1024), (70001, 300), (300000, 1)])
def test_group(m, g):
    gen = torch.Generator(device=DEV).manual_seed(m)
    ids = torch.randint(-2, g + 2, (m,), generator=gen, device=DEV, dtype=torch.int32)
    ids[torch.rand(m, generator=gen, device=DEV) < 0.3] = g // 2          # one adapter with many rows
    for ids in (ids, torch.full_like(ids, -1), torch.full_like(ids, g - 1), torch.full_like(ids, -(2 ** 31))):
        sizes, order = gg.lora_group(ids, g)
        key = torch.where((ids < 0) | (ids >= g), g, ids).long()
        assert torch.equal(order.long(), torch.argsort(key, stable=True))
        assert torch.equal(sizes.long(), torch.bincount(key, minlength=g + 1)[:g])
    wide = key.clone()
    wide[0] = 2 ** 32                                                     # not adapter 0
    sizes, order = gg.lora_group(wide, g)
    assert int(sizes.sum()) == int((wide < g).sum())


def test_group_without_rows():
    sizes, order = gg.lora_group(torch.empty(0, dtype=torch.int32, device=DEV), 5)
    assert torch.all(sizes == 0) and order.numel() == 0


@pytest.mark.parametrize("m", [300, 6000])
@pytest.mark.parametrize("order", [False, True])
def test_in_place_and_rows_without_an_adapter(order, m):
    """out may be base: rows past the last group stay bit for bit, also as a copy; their t is zero."""
    d = make(m, 256, 264, 3, 16, [m - 200, 0, 77], order, 5)
    base, end = d["base_n"], m - 123
    rows = d["order"].long() if order else torch.arange(m, device=DEV)
    base[rows[end:]] = torch.tensor([float("nan"), -0.0, float("inf")], dtype=torch.bfloat16, device=DEV).repeat(88)
    out, t = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], base)
    assert torch.equal(out.view(torch.int16)[rows[end:]], base.view(torch.int16)[rows[end:]])
    assert torch.all(t[end:] == 0)
    same = base.clone()
    got, _ = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], same, out=same)
    assert got is same and torch.equal(same.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("more", [0, 5000])
def test_a_row_keeps_its_nan_to_itself(more):
    """A NaN or infinity in a row, an adapter or a scale reaches that row's, adapter's outputs alone."""
    m = 200 + more
    d = make(m, 136, 72, 3, 8, [90, 0, 100 + more], True, 6)
    clean, clean_t = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"])
    rows = d["order"].long()
    d["x"][rows[3], 5], d["x"][rows[130], 7] = float("nan"), float("inf")
    d["x"][rows[m - 5]] = float("nan")                        # no adapter: not read
    d["down"][1], d["up"][1] = float("nan"), float("inf")     # an adapter without rows
    out, t = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"])
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[[3, 130]] = False
    assert torch.equal(t[keep], clean_t[keep]) and torch.equal(out[rows[keep]], clean[rows[keep]])
    assert torch.isnan(out[rows[3]]).all() and torch.isnan(t[3]).all()
    # infinities of both signs meet in most of the second product's sums: NaN where they do, else infinite
    assert torch.isinf(t[130]).all()
    terms = t[130].double().unsqueeze(1) * d["up"][2].double()
    want = torch.where((terms > 0).all(0) | (terms < 0).all(0), terms[0], float("nan"))
    got = out[rows[130]].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("m", [100, 5000])
def test_bad_order_entries_count_as_none(m):
    """An entry outside [0, M) is skipped: its row is not written and adds nothing to the gradients."""
    sizes = [50, m - 60]
    d = make(m, 64, 64, 2, 8, sizes, True, 7)
    bad = d["order"].clone()
    bad[10], bad[60], bad[m - 5] = -1, m, 2 ** 31 - 1
    out = torch.full((m, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    gg.rdot_lora_forward(d["x"], d["down"], d["up"], d["sizes"], out, order=bad, scale=d["scale"], base=d["base_n"])
    ref, _, tol, _ = reference(d["x"], d["down"], d["up"], sizes, d["order"], d["scale"], d["base_n"])
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[d["order"][[10, 60, m - 5]].long()] = False
    close(out[keep], ref[keep], tol[keep])
    assert torch.all(out[~keep] == 7)
    t = d["dy"][:, :8].contiguous()
    want = t.clone()
    want[[10, 60]] = 0
    t[[10, 60]] = float("nan")
    for z, zs in ((d["x"], None), gg.quantize_mxfp8(d["x"])):
        assert torch.equal(gg.lora_grad_weight(t, z, d["sizes"], bad, zs), gg.lora_grad_weight(want, z, d["sizes"], d["order"], zs))


@pytest.mark.parametrize("more", [0, 7000])
def test_same_result_every_time(more):
    d = make(1000 + more, 2048, 1408, 5, 64, [300, 1, 0, 500 + more, 150], True, 8)
    a = [gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"]) for _ in range(5)]
    w = [gg.lora_grad_weight(a[0][1], d["dy"], d["sizes"], d["order"]) for _ in range(5)]
    for i in range(1, 5):
        assert torch.equal(a[0][0], a[i][0]) and torch.equal(a[0][1], a[i][1]) and torch.equal(w[0], w[i])


def test_strided_and_64_bit_inputs():
    """The calls take strided tensors and int64 sizes and orders; what a row of a wider tensor holds besides is
    not read."""
    d = make(70, 64, 64, 2, 8, [40, 20], True, 9)
    wide = torch.full((70, 200), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:72] = d["x"]
    ref = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"])
    got = gg.lora_forward(wide[:, 8:72], d["down"].transpose(1, 2).contiguous().transpose(1, 2), d["up"], d["sizes"].long(),
                          d["order"].long(), d["scale"].double(), d["base_n"].t().contiguous().t())
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert torch.equal(gg.lora_grad_weight(ref[1], wide[:, 8:72], d["sizes"].long(), d["order"].long()),
                       gg.lora_grad_weight(ref[1], d["x"], d["sizes"], d["order"]))


@pytest.mark.parametrize("m", [2100, 4200])
def test_more_than_32_bits_of_offsets(m):
    """Rows behind the 2^32nd byte and the 2^31st element of x, out and dw."""
    k, r, g = 1 << 20, 8, 2
    gen = torch.Generator(device=DEV).manual_seed(10)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    x[-3:] = randn(gen, (3, k))
    down, up = randn(gen, (g, r, k), 2.0 ** -10), randn(gen, (g, r, 64))
    sizes = [m - 3, 3]
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    out, t = gg.lora_forward(x, down, up, gs)
    ref, ref_t, tol, tol_t = reference(x[-3:], down[1:], up[1:], [3], None, None, None)
    close(t[-3:], ref_t, tol_t)
    close(out[-3:], ref, tol)
    assert torch.all(out[:-3] == 0)
    dy = torch.zeros((m, 64), dtype=torch.bfloat16, device=DEV)
    dy[-3:] = out[-3:]
    dx, dt = gg.lora_grad_input(dy, down, up, gs)
    ref, ref_t, tol, tol_t = reference(dy[-3:], up[1:], down[1:], [3], None, None, None)
    close(dx[-3:], ref, tol)
    dw = gg.lora_grad_weight(t, x, gs)
    tg, zg = t[-3:].double(), x[-3:].double()
    close(dw[1], tg.t() @ zg, 6 * U * (tg.abs().t() @ zg.abs()) + U * (tg.t() @ zg).abs())
    assert torch.all(dw[0] == 0)


@pytest.mark.parametrize("more", [0, 4000])
def test_two_streams_at_once(more):
    """Calls hold no shared workspace: the same shapes on two streams at once give the same results."""
    ds = [make(600 + more, 1024, 1408, 4, 32, [100, 200, 0, 250 + more], True, s) for s in (11, 12)]
    run = lambda d, s: gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"], stream=s)
    refs = [run(d, None) for d in ds]
    refs_w = [gg.lora_grad_weight(r[1], d["dy"], d["sizes"], d["order"]) for r, d in zip(refs, ds)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = [run(d, s) for d, s in zip(ds, streams)]
        ws = [gg.lora_grad_weight(o[1], d["dy"], d["sizes"], d["order"], stream=s) for o, d, s in zip(outs, ds, streams)]
        torch.cuda.synchronize()
        for o, r, w, rw in zip(outs, refs, ws, refs_w):
            assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1]) and torch.equal(w, rw)


def test_threads_with_different_groups():
    """Host threads call with few and many groups at once, each on its own stream."""
    import threading
    failed = []

    def work(i, g):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gen = torch.Generator(device=DEV).manual_seed(100 + i)
                ids = torch.randint(-1, g, (300,), generator=gen, device=DEV, dtype=torch.int32)
                t, z = randn(gen, (300, 8)), randn(gen, (300, 64))
                key = torch.where(ids < 0, g, ids).long()
                want = None
                for _ in range(40):
                    sizes, order = gg.lora_group(ids, g, stream=stream)
                    dw = gg.lora_grad_weight(t, z, sizes, order, stream=stream)
                    want = dw if want is None else want
                    if not (torch.equal(order.long(), torch.argsort(key, stable=True)) and torch.equal(dw, want)):
                        failed.append((g, "another result"))
        except Exception as e:   # a thread's exception would be lost
            failed.append((g, repr(e)))

    threads = [threading.Thread(target=work, args=(i, g)) for i, g in enumerate((1, 1024, 17, 600))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_row_numbers_past_32_bits():
    """An int64 entry of the order that 32 bits do not hold counts as none, not as the row of its low bits."""
    d = make(40, 64, 64, 1, 8, [40], True, 30)
    row = int(d["order"][3])
    wide = d["order"].long()
    wide[3] = 2 ** 32 + int(d["order"][5])
    out = torch.full((40, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], wide, d["scale"], d["base_n"], out=out)
    ref = gg.lora_forward(d["x"], d["down"], d["up"], d["sizes"], d["order"], d["scale"], d["base_n"])[0]
    keep = torch.arange(40, device=DEV) != row
    assert torch.equal(out[keep], ref[keep]) and torch.all(out[row] == 7)


@pytest.mark.parametrize("m", [130, 5000])
def test_captured_step_follows_its_inputs(m):
    """A captured group + forward + gradients replays with other ids, rows and sizes than it was captured with, on
    a grid that its shapes alone decide."""
    k, n, g, r = 256, 384, 6, 16
    d = make(m, k, n, g, r, [0] * g, False, 13)
    ids = torch.zeros(m, dtype=torch.int32, device=DEV)

    def step():
        sizes, order = gg.lora_group(ids, g)
        zq, zs = gg.quantize_mxfp8(d["x"])
        out, t = gg.lora_forward(d["x"], d["down"], d["up"], sizes, order, d["scale"], d["base_n"])
        dx, dt = gg.lora_grad_input(d["dy"], d["down"], d["up"], sizes, order, d["scale"], d["base_k"])
        return out, dx, gg.lora_grad_weight(t, d["dy"], sizes, order), gg.lora_grad_weight(dt, zq, sizes, order, zs)

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = step()
    gen = torch.Generator(device=DEV).manual_seed(14)
    for spread in (1, 2, 9):
        ids.copy_(torch.randint(0, spread, (m,), generator=gen, device=DEV))
        d["x"].copy_(randn(gen, (m, k)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m", [333, 5000])
def test_a_training_step_of_a_projection(m):
    """The calls together, as a frozen projection with adapters trains: forward beside the projection, the input
    kept in 8 bits, the backward pass through both, against autograd in 64 bits. The adapters' gradients see the
    kept input, so the 64-bit gradient of down takes the checkpoint's values. Errors of t and dt, rounded to bf16
    for the gradients, are H of them."""
    k, n, g, r = 288, 416, 5, 24
    d = make(m, k, n, g, r, [0] * g, False, 15)
    gen = torch.Generator(device=DEV).manual_seed(16)
    ids = torch.randint(-1, g, (m,), generator=gen, device=DEV, dtype=torch.int32)
    w = randn(gen, (1, k, n), k ** -0.5)
    one = torch.tensor([m], dtype=torch.int32, device=DEV)
    sizes, order = gg.lora_group(ids, g)
    base = gg.ragged_dot(d["x"], w, one)
    y, t = gg.lora_forward(d["x"], d["down"], d["up"], sizes, order, d["scale"], base, out=base)
    kept = gg.quantize_mxfp8(d["x"])
    dbase = gg.grad_input(d["dy"], w, one)
    dx, dt = gg.lora_grad_input(d["dy"], d["down"], d["up"], sizes, order, d["scale"], dbase, dx=dbase)
    dup = gg.lora_grad_weight(t, d["dy"], sizes, order)
    ddown = gg.lora_grad_weight(dt, kept[0], sizes, order, kept[1])

    x, w64 = d["x"].double().requires_grad_(), w[0].double()
    down, up, scale = d["down"].double().requires_grad_(), d["up"].double().requires_grad_(), d["scale"].double()
    live = (ids >= 0).double().unsqueeze(1)
    i = ids.clamp(min=0).long()
    t64 = torch.einsum("mk,mrk->mr", x, down[i]) * scale[i].unsqueeze(1) * live
    y64 = x @ w64 + torch.einsum("mr,mrn->mn", t64, up[i])
    y64.backward(d["dy"].double())
    # values: two roundings to bf16 (the projection's, the sum's) and the sums' own errors
    mag = x.detach().abs() @ w64.abs()
    tm = (x.detach().abs().unsqueeze(1) * down.detach()[i].abs()).sum(2) * scale[i].abs().unsqueeze(1) * live
    ym = mag + torch.einsum("mr,mrn->mn", tm, up.detach()[i].abs())
    close(y, y64.detach(), H * (x.detach() @ w64).abs() + H * (1 + H) * y64.detach().abs() + (2 * (k + 2 * r) * U + H * H) * ym)
    dy64 = d["dy"].double()
    dt64 = torch.einsum("mn,mrn->mr", dy64, up.detach()[i]) * scale[i].unsqueeze(1) * live
    dtm = torch.einsum("mn,mrn->mr", dy64.abs(), up.detach()[i].abs()) * scale[i].abs().unsqueeze(1) * live
    dxm = dy64.abs() @ w64.abs().t() + torch.einsum("mr,mrk->mk", dtm, down.detach()[i].abs())
    close(dx, x.grad, H * (dy64 @ w64.t()).abs() + H * (1 + H) * x.grad.abs() + (2 * (n + 2 * r) * U + H * H) * dxm)
    xq = _mxfp8.decode(*kept)
    onehot = torch.nn.functional.one_hot(i, g).double() * live
    ref = torch.einsum("mg,mr,mk->grk", onehot, dt64, xq)
    tol = torch.einsum("mg,mr,mk->grk", onehot, H * dt64.abs() + 2 * (n + m + 2) * U * dtm, xq.abs())
    close(ddown, ref, tol)
    tol = torch.einsum("mg,mr,mn->grn", onehot, H * t64.detach().abs() + 2 * (k + m + 2) * U * tm, dy64.abs())
    close(dup, up.grad, tol)
    # and down's own gradient, of the unrounded input: the checkpoint is off by 2^-4 of an element at most, or
    # by half its smallest step, 2^-10 of the scale (a block's largest is above 224 of it)
    blockmax = x.detach().abs().unflatten(1, (-1, 32)).amax(2).repeat_interleave(32, 1)
    off = 2.0 ** -4 * x.detach().abs() + 2.0 ** -10 / 224 * blockmax
    tol = torch.einsum("mg,mr,mk->grk", onehot, dt64.abs(), off) + torch.einsum(
        "mg,mr,mk->grk", onehot, H * dt64.abs() + 2 * (n + m + 2) * U * dtm, xq.abs())
    close(ddown, down.grad, tol)


def test_gradients_are_differences_of_the_forward():
    """The analytic gradients against central differences of the 64-bit forward along random directions."""
    m, k, n, g, r = 40, 64, 96, 3, 8
    d = make(m, k, n, g, r, [15, 0, 20], True, 17, base=False)
    sizes = [15, 0, 20]
    gs, order, scale = d["sizes"], d["order"], d["scale"]
    loss = lambda x, down, up: float((reference(x, down, up, sizes, order, scale, None)[0] * d["dy"].double()).sum())
    _, t = gg.lora_forward(d["x"], d["down"], d["up"], gs, order, scale)
    dx, dt = gg.lora_grad_input(d["dy"], d["down"], d["up"], gs, order, scale)
    grads = (dx, gg.lora_grad_weight(dt, d["x"], gs, order), gg.lora_grad_weight(t, d["dy"], gs, order))
    at = [d["x"].double(), d["down"].double(), d["up"].double()]
    gen = torch.Generator(device=DEV).manual_seed(18)
    for which in range(3):
        v = torch.randn(at[which].shape, generator=gen, device=DEV, dtype=torch.float64)
        eps = 1e-3                           # the loss is linear in each: the difference has no error of its own
        hi, lo = list(at), list(at)
        hi[which], lo[which] = at[which] + eps * v, at[which] - eps * v
        diff = (loss(*hi) - loss(*lo)) / (2 * eps)
        got = float((grads[which].double() * v).sum())
        # each gradient element is off by about H of the terms it sums: bounded by their absolute sum
        bound = 3 * H * float((grads[which].double().abs() * v.abs()).sum()) + 3 * H * float(grads[which].abs().max()) * v.abs().sum() * 0.1
        assert abs(got - diff) <= float(bound)


def test_a_wait_limit_stops_the_call_and_is_reported():
    """A limit of a nanosecond makes waits run out: the calls end early, free what they hold and set the device's status
    bit, which stays until it is cleared; the next calls are right. The few-row form has no such waits."""
    d = make(5000, 2048, 1408, 3, 64, [3000, 0, 1900], True, 19)
    args = (d["down"], d["up"], d["sizes"], d["order"], d["scale"])
    gg.rdot_lora_clear_status()
    ref = gg.lora_forward(d["x"], *args, d["base_n"])
    codes = gg.quantize_mxfp8(d["x"])
    ref_w = [gg.lora_grad_weight(ref[1], d["dy"], d["sizes"], d["order"]), gg.lora_grad_weight(ref[1], codes[0], d["sizes"], d["order"], codes[1])]
    assert gg.rdot_lora_read_status() == 0
    calls = (lambda: gg.lora_forward(d["x"], *args, d["base_n"]), lambda: gg.lora_forward(d["x"], *args[:3], scale=d["scale"]),
             lambda: gg.lora_grad_weight(ref[1], d["dy"], d["sizes"], d["order"]),
             lambda: gg.lora_grad_weight(ref[1], codes[0], d["sizes"], d["order"], codes[1]),
             lambda: gg.lora_grad_weight(ref[1], d["dy"], d["sizes"]))
    try:
        for call in calls:
            gg.rdot_lora_set_wait_timeout(1)
            call()
            assert gg.rdot_lora_read_status() == gg.RDOT_STATUS_BIT_TIMEOUT
            gg.rdot_lora_set_wait_timeout(0)
            call()
            assert gg.rdot_lora_read_status() == gg.RDOT_STATUS_BIT_TIMEOUT     # sticky
            gg.rdot_lora_clear_status()
            assert gg.rdot_lora_read_status() == 0
    finally:
        gg.rdot_lora_set_wait_timeout(0)
    again = gg.lora_forward(d["x"], *args, d["base_n"])
    assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])
    assert torch.equal(calls[2](), ref_w[0]) and torch.equal(calls[3](), ref_w[1])
    assert gg.rdot_lora_read_status() == 0
