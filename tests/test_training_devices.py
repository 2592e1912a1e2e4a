"""Calls launch on their tensors' device and stream, whichever device is
current (CPU: tensors that say they are on a second device, a library that
records where it is called)."""
import contextlib
import types

import pytest
import torch

from ring_allreduce_virtual_gb300 import training


class OnSecond(torch.Tensor):
    is_cuda = True
    device = torch.device("cpu")  # where the allocations of this test go

    def get_device(self):
        return 1


def tensor(*shape):
    return torch.zeros(*shape).as_subclass(OnSecond)


class Library:
    def __init__(self, state):
        self.state, self.calls = state, []

    def __getattr__(self, name):
        def call(*args):
            if "Workspace" not in name:
                self.calls.append((name, self.state["device"], args[-1]))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    state = {"device": 0, "stream": None}
    lib = Library(state)

    @contextlib.contextmanager
    def device(index):
        was, state["device"] = state["device"], index
        yield
        state["device"] = was

    @contextlib.contextmanager
    def stream(s):
        was = dict(state)
        state.update(device=s.device_index, stream=s)
        yield
        state.update(was)

    monkeypatch.setattr(training.vr, "lib", lambda: lib)
    monkeypatch.setattr(training, "_raw_stream", lambda i: state["stream"].handle if state["stream"] else 100 + i)
    monkeypatch.setattr(training, "_current_device", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    lib.enter = device
    training._backward_workspace.cache_clear()
    yield lib
    training._backward_workspace.cache_clear()


def calls(**kw):
    x, m = tensor(2, 8), tensor(2)
    yield "vrLayerNormForward", lambda: training.layer_norm_forward(x, **kw)
    yield "vrLayerNormBackward", lambda: training.layer_norm_backward(x, x, m, m, **kw)
    yield "vrGradNorm", lambda: training.grad_norm([x, m], **kw)
    yield "vrGradNorm", lambda: training.grad_norm(training.TensorList([x, m]), **kw)
    yield "vrClipGradNorm", lambda: training.clip_grad_norm([x, m], 1.0, **kw)


@pytest.mark.parametrize("current", [0, 1])
def test_launches_on_the_tensors_device(library, current):
    with library.enter(current):
        for name, call in calls():
            call()
            assert library.calls[-1] == (name, 1, 101)
            assert library.state["device"] == current


def test_launches_on_a_given_stream(library):
    for name, call in calls(stream=types.SimpleNamespace(device_index=1, handle=77)):
        call()
        assert library.calls[-1] == (name, 1, 77)
        assert library.state["device"] == 0


def test_streams_of_another_device_are_refused(library):
    for _, call in calls(stream=types.SimpleNamespace(device_index=0, handle=77)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not library.calls
