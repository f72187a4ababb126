"""Results of calls on a stream that is not the current one are allocated on that stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def specv():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    import speculative_decoding_verification_specv_gb300 as m
    m.load(build_if_missing=True)
    return m


def _stream_of(t):
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not of the allocator")


@pytest.mark.parametrize("given", [True, False], ids=["given", "current"])
def test_results_are_allocated_on_the_stream_of_the_call(specv, given):
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn((4, 3, 2501), generator=g, device=DEV)
    x = torch.randint(0, 2501, (4, 3), generator=g, device=DEV, dtype=torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = side if given else None
    want = side.cuda_stream if given else torch.cuda.current_stream().cuda_stream
    lp = specv.token_logprobs(z, x, top_n=3, stream=s)
    grad = specv.token_logprobs_backward(z, x, lp.stats, lp.entropy, lp.logprobs, stream=s)
    loss, dq = specv.distill(z, z, stream=s)
    norm = specv.clip_grads([z], float("inf"), stream=s)
    nothing = specv.clip_grads([], 1.0, stream=s)
    torch.cuda.synchronize()
    for t in (*lp, grad, loss, dq, norm, nothing):
        assert _stream_of(t) == want
    # the caller's own tensors stay where they are
    out = torch.empty_like(z)
    assert specv.token_logprobs_backward(z, x, lp.stats, lp.entropy, lp.logprobs, out=out,
                                         stream=s) is out
    torch.cuda.synchronize()
    assert torch.equal(out, grad)
