"""Host-side argument checks of the routing gradients: they answer without a GPU, and a refused call
touches no pointer."""
import ctypes

import pytest

import group_gemm_gb300 as gg

P = ctypes.c_void_p(1 << 20)      # aligned, never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 2)
OK, INVALID, UNSUPPORTED = gg.RDOT_OK, gg.RDOT_ERR_INVALID_ARG, gg.RDOT_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    gg.build()
    return gg.load()


@pytest.mark.parametrize("ptrs, t, k, n, status", [
    ([P] * 7, -1, 2, 16, INVALID),
    ([P] * 7, 4, 0, 16, INVALID),
    ([P] * 7, 4, 2, 0, INVALID),
    ([P] * 7, 4, 2, 12, UNSUPPORTED),                    # rows of 16-byte vectors
    ([P] * 7, 4, 2, 1 << 40, UNSUPPORTED),
    ([P] * 7, 1 << 30, 2, 16, UNSUPPORTED),              # T*k = 2^31
    ([P] * 7, 1 << 62, 4, 16, UNSUPPORTED),              # T*k overflows 64 bits
    ([None] * 7, 0, 2, 16, OK),                          # no tokens: nothing to do
    *[([None if i == j else P for i in range(7)], 4, 2, 16, INVALID) for j in range(7)],
    *[([ODD if i == j else P for i in range(7)], 4, 2, 16, INVALID) for j in range(7)],
])
def test_unpermute_grad_refusals(lib, ptrs, t, k, n, status):
    dout, y, order, inv, w, dy, dw = ptrs
    assert lib.rdot_moe_unpermute_grad(dout, y, order, inv, w, t, k, n, dy, dw, None) == status


@pytest.mark.parametrize("ptrs, dtype, t, k, n, status", [
    ([P] * 3, gg.RDOT_E4M3, 4, 2, 16, INVALID),
    ([P] * 3, gg.RDOT_F32, -1, 2, 16, INVALID),
    ([P] * 3, gg.RDOT_F32, 4, 0, 16, INVALID),
    ([P] * 3, gg.RDOT_F32, 4, 2, 0, INVALID),
    ([P] * 3, gg.RDOT_F32, 4, 2, 6, UNSUPPORTED),
    ([P] * 3, gg.RDOT_BF16, 4, 2, 12, UNSUPPORTED),
    ([P] * 3, gg.RDOT_BF16, 1 << 30, 2, 16, UNSUPPORTED),
    ([P] * 3, gg.RDOT_F32, 4, 2, 1 << 40, UNSUPPORTED),
    ([None] * 3, gg.RDOT_F32, 0, 2, 12, OK),
    *[([None if i == j else P for i in range(3)], gg.RDOT_BF16, 4, 2, 16, INVALID) for j in range(3)],
    *[([ODD if i == j else P for i in range(3)], gg.RDOT_BF16, 4, 2, 16, INVALID) for j in range(3)],
])
def test_permute_grad_refusals(lib, ptrs, dtype, t, k, n, status):
    dxs, inv, dx = ptrs
    assert lib.rdot_moe_permute_grad(dxs, dtype, inv, t, k, n, dx, None) == status


@pytest.mark.parametrize("ptrs, dtype, t, e, k, mode, status", [
    ([P] * 5, gg.RDOT_E4M3, 4, 8, 2, 0, INVALID),
    ([P] * 5, gg.RDOT_F32, -1, 8, 2, 0, INVALID),
    ([P] * 5, gg.RDOT_F32, 4, 8, 9, 0, INVALID),                     # k above E
    ([P] * 5, gg.RDOT_F32, 4, 8, 2, 3, INVALID),                     # unknown weight mode
    ([P] * 5, gg.RDOT_F32, 4, 40, 33, 0, UNSUPPORTED),               # k above the 32 a warp holds
    ([P] * 5, gg.RDOT_F32, 4, gg.RDOT_MAX_GROUPS + 1, 2, 0, UNSUPPORTED),
    ([P] * 5, gg.RDOT_F32, 1 << 40, 8, 2, 0, UNSUPPORTED),
    ([None] * 5, gg.RDOT_BF16, 0, 8, 2, 1, OK),
    ([None, P, P, P, P], gg.RDOT_F32, 4, 8, 2, gg.RDOT_ROUTER_SOFTMAX, INVALID),   # that mode reads the logits
    *[([None if i == j else P for i in range(5)], gg.RDOT_F32, 4, 8, 2, 0, INVALID) for j in range(1, 5)],
    *[([ODD if i == j else P for i in range(5)], gg.RDOT_F32, 4, 8, 2, 1, INVALID) for j in range(5)],
])
def test_router_topk_grad_refusals(lib, ptrs, dtype, t, e, k, mode, status):
    logits, ids, w, dw, dl = ptrs
    assert lib.rdot_router_topk_grad(logits, dtype, ids, w, dw, t, e, k, mode, dl, None) == status


def test_high_level_calls_check_shapes_and_types():
    import torch
    bf = torch.zeros((4, 16), dtype=torch.bfloat16)
    ids = torch.zeros((2, 2), dtype=torch.int32)
    w = torch.zeros((2, 2))
    with pytest.raises(TypeError):
        gg.moe_unpermute_grad(torch.zeros((2, 16)), bf, ids.view(-1), ids.view(-1), w)
    with pytest.raises(ValueError):
        gg.moe_unpermute_grad(bf[:2, :8], bf, ids.view(-1), ids.view(-1), w)
    with pytest.raises(ValueError):
        gg.moe_unpermute_grad(bf[:2], bf, ids.view(-1)[:3], ids.view(-1), w)
    with pytest.raises(ValueError):
        gg.moe_permute_grad(bf, ids.view(-1), 3)
    with pytest.raises(ValueError):
        gg.moe_permute_grad(bf, ids.view(-1)[:2], 2)
    with pytest.raises(ValueError):
        gg.router_topk_grad(torch.zeros((2, 8)), ids, w, w[:1])
    with pytest.raises(TypeError):
        gg.rdot_router_topk_grad(None, ids, w, w, 0, torch.zeros((2, 8), dtype=torch.float16), stream=0)


def test_raw_calls_refuse_two_element_sizes():
    """The element size is taken from one tensor and used for the other."""
    import torch
    ids = torch.zeros((2, 2), dtype=torch.int32)
    w = torch.zeros((2, 2))
    with pytest.raises(TypeError):
        gg.rdot_router_topk_grad(torch.zeros((2, 8), dtype=torch.bfloat16), ids, w, w, gg.RDOT_ROUTER_SOFTMAX,
                                 torch.zeros((2, 8)), stream=0)
    with pytest.raises(TypeError):
        gg.rdot_moe_permute_grad(torch.zeros((4, 16)), ids.view(-1), torch.zeros((2, 16), dtype=torch.bfloat16), stream=0)
