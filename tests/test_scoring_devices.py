"""The device that token_logprobs, its gradient, distill and clip_grads are called on,
without a GPU: tensors that say they are on cuda:1 while cuda:0 is current, a stand-in
for the library that notes the device current at the call, and streams of either device."""
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_verification_specv_gb300 as specv
from speculative_decoding_verification_specv_gb300 import scoring


class OnSecond(torch.Tensor):
    """A tensor in host memory that calls itself one of cuda:1."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


def _second(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnSecond)


@pytest.fixture
def calls(monkeypatch):
    """(entry point, device current at the call, stream handle) of every library call."""
    state = SimpleNamespace(current=0, calls=[])

    class Device:
        def __init__(self, dev):
            self.index = torch.device(dev).index

        def __enter__(self):
            self.before, state.current = state.current, self.index

        def __exit__(self, *exc):
            state.current = self.before

    class Stream(Device):  # the context of torch.cuda.stream
        def __init__(self, stream):
            super().__init__(stream.device)
            self.stream = stream

        def __enter__(self):
            super().__enter__()
            state.stream = self.stream

        def __exit__(self, *exc):
            super().__exit__(*exc)
            state.stream = None

    state.stream = None

    def raw_stream(index):
        return 1000 + index if state.stream is None else state.stream.cuda_stream

    def entry(name):
        def call(*args):
            state.calls.append((name, state.current, args[-1]))
            return 0
        return call

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw_stream, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(scoring, "_entry", entry)
    monkeypatch.setattr(scoring, "_empty",
                        lambda shape, dtype, device: torch.zeros(shape, dtype=dtype).as_subclass(OnSecond))
    monkeypatch.setattr(scoring, "_table", lambda tensors, name: (
        [t.data_ptr() for t in tensors], [t.numel() for t in tensors], [0] * len(tensors)))
    return state


def _every_call(stream):
    z, x, f = _second(2, 3, 8), _second(2, 3, dtype=torch.int32), _second(2, 3)
    return [("specv_token_logprobs", lambda: specv.token_logprobs(z, x, 2, stream)),
            ("specv_token_logprobs_backward",
             lambda: specv.token_logprobs_backward(z, x, _second(2, 3, 2), f, f, stream=stream)),
            ("specv_distill", lambda: specv.distill(z, _second(2, 3, 8), f, stream=stream)),
            ("specv_clip_grads", lambda: specv.clip_grads([z], 1.0, stream=stream))]


def test_calls_are_made_on_the_tensors_device(calls):
    for name, call in _every_call(None):
        call()
        assert calls.calls.pop() == (name, 1, 1001) and not calls.calls and calls.current == 0


def test_a_stream_of_the_tensors_device_is_taken(calls):
    mine = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)
    for name, call in _every_call(mine):
        call()
        assert calls.calls.pop() == (name, 1, 77) and not calls.calls and calls.current == 0


def test_a_stream_of_another_device_is_refused(calls):
    other = SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=78)
    for _, call in _every_call(other):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not calls.calls and calls.current == 0
