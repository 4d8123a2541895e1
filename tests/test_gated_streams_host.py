"""A given stream belongs to the tensors' device, whatever device is current (on
the CPU, with stand-ins for streams and for tensors of a second device)."""
import contextlib

import pytest
import torch

from selective_state_space_39_b200 import _binding as bnd

ONE = torch.device("cuda", 1)


class OnOne(torch.Tensor):
    is_cuda = True
    device = ONE


class Stream:
    def __init__(self, device):
        self.device = device


@pytest.fixture
def call(monkeypatch):
    """A call that answers with the stream that it runs under."""
    current = []

    def external(pointer, device=None):
        s = Stream(device if device is not None else torch.device("cuda", 0))  # the current device
        s.pointer = pointer
        return s

    @contextlib.contextmanager
    def under(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "stream", under)
    return bnd._streamed(lambda *t, **kw: current[-1] if current else None)


def tensor():
    return torch.zeros(1).as_subclass(OnOne)


def test_another_library_s_stream_is_one_of_the_tensors_device(call):
    class Foreign:
        cuda_stream = 77

    for args, kw in (((tensor(),), {}), ((), {"x": tensor()}), ((None, torch.zeros(1), tensor()), {})):
        s = call(*args, stream=Foreign(), **kw)
        assert s.pointer == 77 and s.device == ONE


def test_a_stream_of_another_device_is_refused(call):
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        call(tensor(), stream=Stream(torch.device("cuda", 0)))
    own = Stream(ONE)
    assert call(tensor(), stream=own) is own
    assert call(tensor()) is None
