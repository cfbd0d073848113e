"""The Python binding's own host code, without a GPU: which stream a call is given."""
import pytest
import torch

import group_gemm_gb300 as gg


class FakeStream:
    cuda_stream = 77


@pytest.fixture
def asked(monkeypatch):
    """The devices torch.cuda.current_stream is asked for."""
    devices = []

    def current_stream(device=None):
        devices.append(device)
        return FakeStream()

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    return devices


@pytest.mark.parametrize("device", [None, 0, "cuda:0", torch.device("cuda")])
def test_the_current_stream_of_any_form_of_device(asked, device):
    assert gg._stream(None, device) == 77 and asked == [device]


def test_given_streams_are_passed_on(asked):
    assert gg._stream(FakeStream(), None) == 77 and gg._stream(5, None) == 5 and asked == []


def test_no_alloc_status_without_a_device(asked):
    """rdot_no_alloc_read_status takes neither a tensor nor (by default) a device."""
    gg.build()
    with pytest.raises(gg.RdotError) as e:
        gg.rdot_no_alloc_read_status(None)
    assert e.value.status == gg.RDOT_ERR_INVALID_ARG and asked == [None]


def bad_outs(m, n, dtype):
    """(an output that does not hold [m, n] of dtype, the error it gets)."""
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    return [(torch.empty((m, n), dtype=other), TypeError),
            (torch.empty((m, n), dtype=torch.uint8), TypeError),
            (torch.empty((m - 1, n), dtype=dtype), ValueError),
            (torch.empty((m, n // 2), dtype=dtype), ValueError),
            (torch.empty((m, 2 * n), dtype=dtype)[:, ::2], ValueError),
            (torch.empty((n, m), dtype=dtype).t(), ValueError),
            (torch.empty((m, n), dtype=dtype, device="meta"), ValueError)]


def test_mxfp4_forward_refuses_outputs_it_cannot_fill():
    m, k, n, g = 4, 64, 64, 2
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    args = (u8(m, k // 2), u8(m, k // 32), u8(g, n, k // 2), u8(g, 1, 1, 512), torch.zeros(g, dtype=torch.int32))
    for out, error in bad_outs(m, n, torch.bfloat16) + [(torch.empty(m * n, dtype=torch.bfloat16), ValueError),
                                                        (torch.empty((m + 1, n), dtype=torch.bfloat16), ValueError)]:
        with pytest.raises(error, match="out must be"):
            gg.ragged_dot_mxfp4(*args, out=out)


def older_calls():
    m, k, n, g, t = 8, 64, 64, 2, 4
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    gs, order, w = torch.zeros(g, dtype=torch.int32), torch.zeros(m, dtype=torch.int32), torch.zeros((t, 2))
    bf16, f32 = torch.bfloat16, torch.float32
    x, y, r = bf(m, k), bf(m, n), bf(g, k, n)
    return {
        "ragged_dot": (lambda out: gg.ragged_dot(x, r, gs, out=out), (m, n), bf16),
        "ragged_dot, fp32 out": (lambda out: gg.ragged_dot(x, r, gs, out_dtype=f32, out=out), (m, n), f32),
        "grad_weight": (lambda out: gg.grad_weight(x, y, gs, out_dtype=f32, dw=out), (g * k, n), f32),
        "grad_input": (lambda out: gg.grad_input(y, r, gs, dlhs=out), (m, k), bf16),
        "ragged_dot_gated": (lambda out: gg.ragged_dot_gated(x, r, r, gs, out=out), (m, n), bf16),
        "grad_weight_mxfp8": (lambda out: gg.grad_weight_mxfp8(u8(m, k), u8(g, k), u8(m, n), u8(g, n), gs, out=out,
                                                               out_dtype=f32), (g * k, n), f32),
        "ragged_dot_combine": (lambda out: gg.ragged_dot_combine(x, r, gs, order, w, out=out), (t, n), f32),
        "moe_unpermute": (lambda out: gg.moe_unpermute(y, order, w, out=out), (t, n), bf16),
        "ragged_dot_mxfp8": (lambda out: gg.ragged_dot_mxfp8(u8(m, k), u8(m, 2), u8(g, k, n), u8(g, 2, n), gs, out=out),
                             (m, n), bf16),
        "padded_ragged_dot": (lambda out: gg.padded_ragged_dot(x, r, gs, 128, out=out), (m, n), bf16),
    }


@pytest.mark.parametrize("name", list(older_calls()))
def test_calls_refuse_outputs_they_cannot_fill(name, monkeypatch):
    """A larger or reshaped contiguous output still does; the call then goes on to its stream."""
    call, (rows, cols), dtype = older_calls()[name]
    for out, error in bad_outs(rows, cols, dtype):
        with pytest.raises(error, match="must be"):
            call(out)

    class Reached(Exception):
        pass

    def run_stream(stream, device):
        raise Reached

    monkeypatch.setattr(gg, "_run_stream", run_stream)
    for out in (None, torch.empty((rows, cols), dtype=dtype), torch.empty((rows + 3, cols), dtype=dtype),
                torch.empty(rows * cols, dtype=dtype)):
        with pytest.raises(Reached):
            call(out)


def two_device_calls():
    """Calls of the MXFP4 product and the routing gradients, and their operands."""
    m, k, n, g, t = 4, 64, 64, 2, 2
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    return {
        "ragged_dot_mxfp4": (gg.ragged_dot_mxfp4, [u8(m, k // 2), u8(m, k // 32), u8(g, n, k // 2), u8(g, 1, 1, 512),
                                                   i32(g)]),
        "moe_unpermute_grad": (gg.moe_unpermute_grad, [bf(t, n), bf(m, n), i32(m), i32(m), torch.zeros((t, 2))]),
        "moe_permute_grad": (lambda dxs, inv: gg.moe_permute_grad(dxs, inv, 2), [bf(m, n), i32(m)]),
        "router_topk_grad": (gg.router_topk_grad, [torch.zeros((t, 8)), i32(t, 2), torch.zeros((t, 2)),
                                                   torch.zeros((t, 2))]),
    }


@pytest.mark.parametrize("name", list(two_device_calls()))
def test_calls_refuse_tensors_of_two_devices(name):
    call, args = two_device_calls()[name]
    for i in range(len(args)):
        with pytest.raises(ValueError, match="one device"):
            call(*[a.to("meta") if j == i else a for j, a in enumerate(args)])
