"""Which workspace the binding gives a call, on the host with a stand-in for
torch: a workspace that is kept must never be recorded in a graph, which would
go on using it after a larger call has replaced it."""

import contextlib

import pytest

from trellis_quantized_linear_rot_gb300 import spec


class Tensor:
    made = 0

    def __init__(self):
        Tensor.made += 1
        self.at = 4096 * Tensor.made

    def data_ptr(self):
        return self.at


class Torch:
    """As much of torch as spec._workspace uses; `capturing` holds the streams
    that are being captured."""

    uint8 = "uint8"

    def __init__(self):
        self.current, self.capturing = "default", set()
        torch = self

        class Cuda:
            @staticmethod
            @contextlib.contextmanager
            def stream(s):
                before, torch.current = torch.current, s
                yield
                torch.current = before

            @staticmethod
            def device(d):
                return contextlib.nullcontext()

            @staticmethod
            def is_current_stream_capturing():
                return torch.current in torch.capturing

        class C:
            _cuda_isCurrentStreamCapturing = staticmethod(Cuda.is_current_stream_capturing)

        self.cuda, self._C = Cuda, C

    def zeros(self, n, dtype, device):
        return Tensor()


class Device:
    index = 0


@pytest.fixture
def torch(monkeypatch):
    t = Torch()
    monkeypatch.setattr(spec, "torch", t)
    monkeypatch.setattr(spec, "_workspaces", {})
    return t


def ask(stream, nbytes=100, handle=7):
    return spec._workspace("x", nbytes, Device, handle, stream)


@pytest.mark.parametrize("stream", [None, "side"])
def test_a_workspace_is_kept_for_a_stream_and_grows(torch, stream):
    a = ask(stream)
    assert ask(stream) is a and ask(stream, 60) is a
    b = ask(stream, 101)
    assert b is not a and ask(stream) is b and ask(stream, handle=8) is not b
    assert torch.current == "default"


@pytest.mark.parametrize("stream", [None, "side"])
def test_a_captured_call_has_its_own(torch, stream):
    kept = ask(stream)
    torch.capturing = {stream or "default"}
    one, two = ask(stream), ask(stream)
    assert len({kept[0], one[0], two[0]}) == 3
    torch.capturing = set()
    assert ask(stream) is kept


def test_it_is_the_calls_own_stream_that_counts(torch):
    """Another stream than the current one is given: what the current one
    does is not asked."""
    kept = ask("side")
    torch.capturing = {"side"}
    assert ask("side") is not kept
    torch.capturing = {"default"}
    assert ask("side") is kept
