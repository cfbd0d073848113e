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
