"""MXFP4 on the host: the plain quantiser of the tests against hand-checked blocks, and the argument
checks of the entry points, which answer without a GPU."""
import ctypes

import pytest
import torch

import group_gemm_gb300 as gg
from tests import _mxfp4 as mx

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
OK, INVALID, UNSUPPORTED = gg.RDOT_OK, gg.RDOT_ERR_INVALID_ARG, gg.RDOT_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    gg.build()
    return gg.load()


def test_plain_quantiser_by_hand():
    x = torch.zeros((4, 32))
    # amax 6 -> scale 2^0: every magnitude, the ties between neighbours (to the even code), saturation
    x[0, :18] = torch.tensor([6, -6, 0.25, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.2500001, 5.000001, 7.9, 4, 3, 1.5, 0.5,
                              -0.0])
    # the same a factor of 2^10 down; amax 7.9 keeps floor(log2) = 2
    x[1] = x[0] * 2.0 ** -10
    x[2, 5] = float("inf")
    codes, s, v = mx.quantize(x)
    want = [7, 15, 0, 8, 2, 2, 4, 4, 6, 6, 1, 7, 7, 6, 5, 3, 1, 8]
    assert codes[0, :18].tolist() == want and codes[1, :18].tolist() == want
    assert s[:, 0].tolist() == [127, 117, 255, 0]
    assert v[0, :6].tolist() == [6, -6, 0, 0, 1, 1] and torch.isnan(v[2]).all() and torch.all(v[3] == 0)
    assert torch.equal(mx.decode(mx.pack(codes), s)[:2], v[:2])
    t = mx.tile_scales(torch.arange(130 * 5).view(1, 130, 5).to(torch.uint8))
    assert t.shape == (1, 2, 2, 512)
    assert t[0, 0, 0, 16 * 5 + 4 * 1 + 2] == (37 * 5 + 2) % 256 and t[0, 1, 1, 16 * 1] == (129 * 5 + 4) % 256


@pytest.mark.parametrize("ptrs, dtype, rows, k, status", [
    ([P] * 4, gg.RDOT_E4M3, 4, 64, INVALID),
    ([P] * 4, gg.RDOT_F32, -1, 64, INVALID),
    ([P] * 4, gg.RDOT_F32, 4, 0, INVALID),
    ([P] * 4, gg.RDOT_F32, 4, 48, UNSUPPORTED),                # blocks of 32
    ([P] * 4, gg.RDOT_F32, 4, 1 << 31, UNSUPPORTED),
    ([P] * 4, gg.RDOT_BF16, 1 << 62, 64, UNSUPPORTED),
    ([None] * 4, gg.RDOT_BF16, 0, 64, OK),
    *[([None if i == j else P for i in range(4)], gg.RDOT_BF16, 4, 64, INVALID) for j in range(3)],
    *[([ODD if i == j else P for i in range(4)], gg.RDOT_BF16, 4, 64, INVALID) for j in (0, 1, 3)],
])
def test_quantize_rows_refusals(lib, ptrs, dtype, rows, k, status):
    x, codes, scales, values = ptrs
    assert lib.rdot_quantize_mxfp4(x, dtype, rows, k, codes, scales, values, None) == status


@pytest.mark.parametrize("ptrs, dtype, g, k, n, status", [
    ([P] * 4, gg.RDOT_E2M1, 2, 64, 64, INVALID),
    ([P] * 4, gg.RDOT_F32, 0, 64, 64, INVALID),
    ([P] * 4, gg.RDOT_F32, 2, 0, 64, INVALID),
    ([P] * 4, gg.RDOT_F32, 2, 64, 0, INVALID),
    ([P] * 4, gg.RDOT_F32, gg.RDOT_MAX_GROUPS + 1, 64, 64, UNSUPPORTED),
    ([P] * 4, gg.RDOT_F32, 2, 48, 64, UNSUPPORTED),
    ([P] * 4, gg.RDOT_F32, 2, 64, 60, UNSUPPORTED),
    ([P] * 4, gg.RDOT_F32, 1024, 1 << 30, 1 << 20, UNSUPPORTED),   # more blocks than a grid has
    *[([None if i == j else P for i in range(4)], gg.RDOT_BF16, 2, 64, 64, INVALID) for j in range(3)],
    *[([ODD if i == j else P for i in range(4)], gg.RDOT_BF16, 2, 64, 64, INVALID) for j in range(4)],
])
def test_quantize_weight_refusals(lib, ptrs, dtype, g, k, n, status):
    w, codes, scales, values = ptrs
    assert lib.rdot_quantize_mxfp4_weight(w, dtype, g, k, n, codes, scales, values, None) == status


def test_weight_scale_bytes(lib):
    assert gg.rdot_mxfp4_weight_scale_bytes(8, 4096, 14336) == 8 * 112 * 32 * 512
    assert gg.rdot_mxfp4_weight_scale_bytes(3, 160, 136) == 3 * 2 * 2 * 512
    b = ctypes.c_size_t()
    assert lib.rdot_mxfp4_weight_scale_bytes(0, 64, 64, ctypes.byref(b)) == INVALID
    assert lib.rdot_mxfp4_weight_scale_bytes(2, 48, 64, ctypes.byref(b)) == UNSUPPORTED
    assert lib.rdot_mxfp4_weight_scale_bytes(2, 64, 64, None) == INVALID


@pytest.mark.parametrize("kw, status", [
    (dict(in_dtype=gg.RDOT_E4M3), UNSUPPORTED),
    (dict(out_dtype=gg.RDOT_F32), UNSUPPORTED),
    (dict(k=48), UNSUPPORTED),
    (dict(n=60), UNSUPPORTED),
    (dict(tile_n=256), UNSUPPORTED),
    (dict(flags=gg.RDOT_FLAG_NO_CTA_PAIR), UNSUPPORTED),
    (dict(flags=gg.RDOT_FLAG_SKINNY | gg.RDOT_FLAG_CTA_PAIR), UNSUPPORTED),
    (dict(flags=gg.RDOT_FLAG_SKINNY | gg.RDOT_FLAG_NO_SKINNY), INVALID),
    (dict(k=0), INVALID), (dict(m=-1), INVALID), (dict(groups=0), INVALID),
])
def test_plan_refusals(lib, kw, status):
    base = dict(m=16, k=64, n=64, groups=2, mode=gg.RDOT_MODE_FORWARD_MXFP4, in_dtype=gg.RDOT_E2M1,
                out_dtype=gg.RDOT_BF16, tile_n=0, flags=0)
    base.update(kw)
    h = ctypes.c_void_p()
    assert lib.rdot_plan(ctypes.byref(gg.Problem(**base)), 0, ctypes.byref(h)) == status and not h.value


def test_forward_without_a_plan_and_high_level_checks(lib):
    assert lib.rdot_forward_mxfp4(None, P, P, P, P, P, P, P, None) == INVALID
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    w, ws = torch.zeros((2, 64, 32), dtype=torch.uint8), torch.zeros((2, 1, 1, 512), dtype=torch.uint8)
    gs = torch.zeros(2, dtype=torch.int32)
    for args in ((q, s[:, :1], w, ws, gs), (q, s, w, ws[:1], gs), (q, s, w, ws, gs[:1]), (q[:, :16], s, w, ws, gs)):
        with pytest.raises(ValueError):
            gg.ragged_dot_mxfp4(*args)
    with pytest.raises(TypeError):
        gg.ragged_dot_mxfp4(q.int(), s, w, ws, gs)
    with pytest.raises(ValueError):
        gg.quantize_mxfp4(torch.zeros(64))
    with pytest.raises(ValueError):
        gg.quantize_mxfp4_weight(torch.zeros((64, 64)))
    with pytest.raises(TypeError):
        gg.rdot_quantize_mxfp4(torch.zeros((2, 64), dtype=torch.float16), q, s)
