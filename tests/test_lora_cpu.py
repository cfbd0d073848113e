"""Host-side argument checks of the low-rank adapters and the 8-bit checkpoints: they answer without a GPU,
and a refused call touches no pointer."""
import ctypes

import pytest
import torch

import group_gemm_gb300 as gg
from tests import _mxfp8

P = ctypes.c_void_p(1 << 20)      # aligned, never dereferenced: the checks fail first
Q = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 2)
OK, INVALID, UNSUPPORTED = gg.RDOT_OK, gg.RDOT_ERR_INVALID_ARG, gg.RDOT_ERR_UNSUPPORTED
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    gg.build()
    return gg.load()


def _each(n, value, skip=()):
    return [[value if i == j else (Q if i == 0 else P) for i in range(n)] for j in range(n) if j not in skip]


SIZES = [                                # m, k, n, groups, rank
    ((-1, 64, 64, 2, 8), INVALID), ((4, 0, 64, 2, 8), INVALID), ((4, 64, 0, 2, 8), INVALID),
    ((4, 64, 64, 0, 8), INVALID), ((4, 64, 64, 2, 0), INVALID), ((4, 64, 64, 2, -8), INVALID),
    ((1 << 31, 64, 64, 2, 8), UNSUPPORTED), ((BIG, 64, 64, 2, 8), UNSUPPORTED),
    ((4, 60, 64, 2, 8), UNSUPPORTED), ((4, 64, 60, 2, 8), UNSUPPORTED),
    ((4, BIG, 64, 2, 8), UNSUPPORTED), ((4, 64, BIG, 2, 8), UNSUPPORTED),
    ((4, 64, 64, gg.RDOT_MAX_GROUPS + 1, 8), UNSUPPORTED),
    ((4, 64, 64, 2, 12), UNSUPPORTED), ((4, 64, 64, 2, gg.RDOT_LORA_MAX_RANK + 8), UNSUPPORTED),
]


@pytest.mark.parametrize("call", ["rdot_lora_forward", "rdot_lora_grad_input"])
def test_apply_refusals(lib, call):
    f = getattr(lib, call)
    good = (4, 64, 64, 2, 8)
    for sizes, status in SIZES:
        assert f(*[P] * 7, *sizes, Q, P, None) == status, sizes
    assert f(*[None] * 7, 0, 64, 64, 2, 8, None, None, None) == OK          # no rows: nothing to do
    # x, down, up, group_sizes, order, scale, base, out, t: the first four and out are needed
    for j in range(9):
        args = [P] * 7 + [Q, P]
        args[j] = None
        if j in (0, 1, 2, 3, 7):
            assert f(*args[:7], *good, *args[7:], None) == INVALID, j
        args[j] = ODD
        assert f(*args[:7], *good, *args[7:], None) == INVALID, j
    assert f(P, Q, Q, Q, Q, Q, Q, *good, P, Q, None) == INVALID              # out is x


def test_grad_weight_refusals(lib):
    f = lib.rdot_lora_grad_weight

    def call(t=P, z=P, zt=gg.RDOT_BF16, zs=P, gs=P, order=P, m=4, width=64, groups=2, rank=8, ot=gg.RDOT_F32, dw=P):
        return f(t, z, zt, zs, gs, order, m, width, groups, rank, ot, dw, None)

    for (m, k, _, groups, rank), status in SIZES:
        if k == 64 and not (m == 4 and groups == 2 and rank == 8):
            assert call(m=m, groups=groups, rank=rank) == status
    for width, status in ((0, INVALID), (60, UNSUPPORTED), (BIG, UNSUPPORTED), (-8, INVALID)):
        assert call(width=width) == status
    assert call(width=1 << 30, groups=1024) == UNSUPPORTED                    # more blocks than a grid holds
    assert call(zt=gg.RDOT_E4M3, width=72) == UNSUPPORTED                     # whole scale blocks
    assert call(zt=gg.RDOT_F32) == INVALID and call(ot=gg.RDOT_E4M3) == INVALID
    for name in ("t", "z", "gs", "dw"):
        assert call(**{name: None}) == INVALID and call(**{name: ODD}) == INVALID
    assert call(order=ODD) == INVALID
    assert call(zt=gg.RDOT_E4M3, zs=None) == INVALID


def test_group_refusals(lib):
    f = lib.rdot_lora_group
    assert f(P, -1, 4, P, P, None) == INVALID
    assert f(P, 4, 0, P, P, None) == INVALID
    assert f(P, 4, gg.RDOT_MAX_GROUPS + 1, P, P, None) == UNSUPPORTED
    assert f(P, 1 << 31, 4, P, P, None) == UNSUPPORTED
    for j in range(3):
        for bad in (None, ODD):
            args = [P] * 3
            args[j] = bad
            assert f(args[0], 4, 4, args[1], args[2], None) == INVALID


def test_status_calls(lib):
    assert lib.rdot_lora_read_status(None, None) == INVALID
    assert lib.rdot_lora_set_wait_timeout(5) == OK and lib.rdot_lora_set_wait_timeout(0) == OK


def test_quantize_refusals(lib):
    q, d = lib.rdot_quantize_mxfp8, lib.rdot_dequantize_mxfp8
    for dtype, rows, k, status in ((gg.RDOT_E4M3, 4, 64, INVALID), (gg.RDOT_F32, -1, 64, INVALID),
                                   (gg.RDOT_F32, 4, 0, INVALID), (gg.RDOT_BF16, 4, 48, UNSUPPORTED),
                                   (gg.RDOT_BF16, 4, 1 << 40, UNSUPPORTED), (gg.RDOT_BF16, BIG, 64, UNSUPPORTED)):
        assert q(P, dtype, rows, k, P, P, None) == status
        assert d(P, P, rows, k, dtype, P, None) == status
    assert q(None, gg.RDOT_F32, 0, 64, None, None, None) == OK
    assert d(None, None, 0, 64, gg.RDOT_F32, None, None) == OK
    for j in range(3):
        args = [P] * 3
        args[j] = None
        assert q(args[0], gg.RDOT_F32, 4, 64, args[1], args[2], None) == INVALID
        assert d(args[0], args[1], 4, 64, gg.RDOT_F32, args[2], None) == INVALID
    assert q(ODD, gg.RDOT_F32, 4, 64, P, P, None) == INVALID and q(P, gg.RDOT_F32, 4, 64, ODD, P, None) == INVALID
    assert d(ODD, P, 4, 64, gg.RDOT_F32, P, None) == INVALID and d(P, P, 4, 64, gg.RDOT_F32, ODD, None) == INVALID


def test_high_level_refusals():
    """Shapes, types and devices are checked before anything is launched (CPU tensors serve)."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    x, down, up, gs = z(6, 64), z(2, 8, 64), z(2, 8, 32), z(2, dtype=torch.int32)
    for bad in (dict(x=z(6, 32)), dict(x=z(64)), dict(down=z(3, 8, 64)), dict(up=z(2, 16, 32)),
                dict(group_sizes=z(3, dtype=torch.int32)), dict(order=z(5, dtype=torch.int32)),
                dict(scale=z(3, dtype=torch.float32)), dict(base=z(6, 64)), dict(out=z(6, 64)), dict(out=z(32, 6).t())):
        with pytest.raises(ValueError):
            gg.lora_forward(**{**dict(x=x, down=down, up=up, group_sizes=gs), **bad})
    for bad in (dict(x=x.float()), dict(down=down.float()), dict(base=z(6, 32).float()),
                dict(out=z(6, 32, dtype=torch.float32))):
        with pytest.raises(TypeError):
            gg.lora_forward(**{**dict(x=x, down=down, up=up, group_sizes=gs), **bad})
    with pytest.raises(ValueError):
        gg.lora_grad_input(x, down, up, gs)                        # rows of K columns where N are due
    with pytest.raises(ValueError):
        gg.lora_forward(x, down, up, gs.to("meta"))
    t = z(6, 8)
    for bad in (dict(z=z(5, 64)), dict(t=z(6)), dict(order=z(7, dtype=torch.int32)), dict(dw=z(2, 64, 8, dtype=torch.float32)),
                dict(z=z(6, 64, dtype=torch.uint8), z_scale=z(6, 3, dtype=torch.uint8)),
                dict(group_sizes=gs.to("meta")), dict(group_sizes=z(2, 1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            gg.lora_grad_weight(**{**dict(t=t, z=x, group_sizes=gs), **bad})
    for bad in (dict(t=t.float()), dict(z=z(6, 64, dtype=torch.uint8)), dict(z_scale=z(6, 2, dtype=torch.uint8)),
                dict(dw=z(2, 8, 64, dtype=torch.int32), out_dtype=torch.float32)):
        with pytest.raises(TypeError):
            gg.lora_grad_weight(**{**dict(t=t, z=x, group_sizes=gs), **bad})
    with pytest.raises(ValueError):
        gg.lora_group(z(2, 3, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        gg.quantize_mxfp8(z(64))
    with pytest.raises(ValueError):
        gg.dequantize_mxfp8(z(4, 64, dtype=torch.uint8), z(4, 64, dtype=torch.uint8))
    with pytest.raises(TypeError):
        gg.dequantize_mxfp8(z(4, 64, dtype=torch.uint8), z(4, 2))


def test_plain_mxfp8_codes_are_e4m3():
    """The tests' own grid is the E4M3 format's, and its rounding the format's, ties to even included."""
    c = torch.arange(256, dtype=torch.uint8)
    ref = c.view(torch.float8_e4m3fn).double()
    got = _mxfp8.decode(c, torch.full((8,), 127, dtype=torch.uint8))
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got[~torch.isnan(ref)], ref[~torch.isnan(ref)])
    x = torch.cat((torch.linspace(-448, 448, 9999), torch.arange(-40, 41) * 2.0 ** -11, torch.zeros(16)))
    x = x[:x.numel() // 31 * 31].view(-1, 31)
    x = torch.cat((x, torch.full((x.shape[0], 1), 448.0)), 1)     # one element of each block fixes the scale at 1
    codes, s, values = _mxfp8.quantize(x)
    assert torch.all(s == 127)
    assert torch.equal(codes, x.to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(values, x.to(torch.float8_e4m3fn).double())
