"""The example that uses verify, token_logprobs, distill and clip_grads together:
fitting the draft lowers the divergence and raises the acceptance."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("fit_draft",
                                                  os.path.join(ROOT, "examples", "fit_draft.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kind", [0, 1], ids=["forward", "reverse"])
def test_fitting_the_draft_raises_acceptance(kind):
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    h = _example().fit(steps=60, batch=64, draft=4, vocab=1001, hidden=64, kind=kind, report=None)
    first = sum(x["alpha"] for x in h[:5]) / 5
    last = sum(x["alpha"] for x in h[-5:]) / 5
    assert all(math.isfinite(v) for x in h for k, v in x.items() if k != "alternatives")
    assert last > first + 0.1, (first, last)
    assert h[-1]["loss"] < h[0]["loss"]
    assert h[-1]["tokens_per_step"] > h[0]["tokens_per_step"]
    # ln p of tokens drawn from p is minus its entropy, on average
    mean = sum(x["logprob"] + x["entropy"] for x in h) / len(h)
    assert abs(mean) < 0.2
