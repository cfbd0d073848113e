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
