"""adamw_step's host side without a GPU (and what sampling shares with it): tensors in host memory that call themselves a GPU's,
and the library's entry replaced by one that notes the call."""
import math
import struct

import pytest
import torch

import speculative_decoding_verification_specv_gb300 as specv
from speculative_decoding_verification_specv_gb300 import optim, sampling


class OnGpu(torch.Tensor):
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape).to(dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    made = []

    def entry(name):
        def call(*args):
            made.append((name, args))
            return 0
        return call

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)
    for module in (optim, sampling):
        monkeypatch.setattr(module, "_entry", entry)
    monkeypatch.setattr(optim, "_get_device", lambda t: t.device.index)
    monkeypatch.setattr(sampling, "_empty",
                        lambda shape, dtype, device: torch.zeros(shape, dtype=dtype).as_subclass(OnGpu))
    return made


def _state(p, masters=None):
    return specv.AdamWState([_t(*x.shape) for x in p], [_t(*x.shape) for x in p], None, masters)


def test_shapes_have_to_agree(calls):
    """A transposed matrix has its weight's size, and would go to the wrong weights."""
    p = [_t(5), _t(3, 4), _t(2, 3, 4)]
    g = [_t(5), _t(3, 4), _t(2, 3, 4)]
    specv.adamw_step(p, g, _state(p), 1, 0.1)
    assert len(calls) == 1
    other = lambda k, i, x: [x if j == i else y for j, y in enumerate(k)]
    st = _state(p)
    half = [p[0], _t(3, 4, dtype=torch.bfloat16), p[2]]
    for call in (lambda: specv.adamw_step(p, other(g, 1, _t(4, 3)), st, 1, 0.1),
                 lambda: specv.adamw_step(p, other(g, 1, _t(12, 1)), st, 1, 0.1),
                 lambda: specv.adamw_step(p, other(g, 2, _t(3, 2, 4)), st, 1, 0.1),
                 lambda: specv.adamw_step(p, g, st._replace(exp_avg=other(st.exp_avg, 1, _t(4, 3))), 1, 0.1),
                 lambda: specv.adamw_step(p, g, st._replace(exp_avg_sq=other(st.exp_avg_sq, 2, _t(6, 4))), 1, 0.1),
                 lambda: specv.adamw_step(half, g, st._replace(masters=[None, _t(4, 3), None]), 1, 0.1)):
        with pytest.raises(ValueError, match="shape"):
            call()
    assert len(calls) == 1
    # the same entries in one dimension are taken, on either side
    specv.adamw_step(p, other(g, 1, _t(12)), st, 1, 0.1)
    specv.adamw_step(other(p, 1, _t(12)), g, st, 1, 0.1)
    specv.adamw_step(half, g, st._replace(masters=[None, _t(12), None]), 1, 0.1)
    assert len(calls) == 4


def test_what_is_written_counts_as_written(calls):
    """In place means in place for autograd too: version counters move."""
    p = [_t(5), _t(3, 4, dtype=torch.bfloat16)]
    masters = [None, _t(3, 4)]
    g = [_t(5), _t(3, 4)]
    before = [x._version for x in (*p, masters[1], *g)]
    specv.adamw_step(p, g, _state(p, masters), 1, 0.1)
    assert [x._version for x in (*p, masters[1])] == [v + 1 for v in before[:3]]
    assert [x._version for x in g] == before[3:]  # read only
    with torch.inference_mode():
        q = [_t(5)]
    specv.adamw_step(q, g[:1], _state(q), 1, 0.1)
    z, u, out = _t(2, 3, 8), _t(2, 3), _t(2, 3, 8)
    before = z._version, out._version
    specv.filter_logits(z, 0.7, out=out)
    specv.sample_tokens(z, u, out_filtered=out)
    assert (z._version, out._version) == (before[0], before[1] + 2)
    specv.filter_logits(z, 0.7, out=z)
    assert z._version == before[0] + 1
    specv.filter_logits(z, 0.7)
    specv.sample_tokens(z, u)
    assert z._version == before[0] + 1


@pytest.mark.parametrize("max_norm,there", [(1.0, 1.0), (0.0, 0.0), (3.4e38, 3.4e38), (1e39, math.inf),
                                            (math.inf, math.inf)])
def test_the_largest_norm_as_it_is_given(calls, max_norm, there):
    p, norm = [_t(5)], _t(1)
    specv.adamw_step(p, [_t(5)], _state(p), 1, 0.1, norm=norm, max_norm=max_norm)
    config = calls.pop()[1][2]
    assert struct.unpack("qqddddPPPfIQ", config)[9] == torch.tensor(there).item()
