"""The `stream` argument of the binding: which stream a handle names, and where missing outputs come from.  Host
logic, no GPU: torch's stream calls and the library's entry points are replaced."""
import contextlib

import pytest
import torch

import fp8_blockwise_scaled_b200 as fb

CPU = torch.device("cpu")


class FakeStream:
    def __init__(self, name):
        self.name, self.device = name, CPU


@pytest.fixture
def streams(monkeypatch):
    """The stream that is current, as torch.cuda.stream sets it; ExternalStream(h) is named by its handle."""
    now = [FakeStream("caller")]

    @contextlib.contextmanager
    def current(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream("default"))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None, raising=False)
    return now


@pytest.mark.parametrize("handle,name", [(0, "default"), (1, "default"), (2, 2), (0x7F00, 0x7F00)])
def test_handle_of_the_default_stream_is_that_stream(streams, handle, name):
    seen = []

    def call():
        seen.append(streams[-1].name)
        return torch.zeros(1)

    fb._on_stream(handle, CPU, call)
    assert seen == [name] and streams[-1].name == "caller"
