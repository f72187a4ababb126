"""Calls of several host threads on one stream: the launches of clip_grads, whose second
one reads what the first leaves in the stream's workspace, and of verify, which uses the
same workspace, do not come between one another's."""
import threading

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


def _gradients(seed, n, size):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(size + 7 * i, generator=g, device=DEV).mul_(10.0 ** (seed - 3))
            for i in range(n)]


def _verify_inputs(B, K, V):
    g = torch.Generator(device=DEV).manual_seed(9)
    zt = torch.randn((B, K + 1, V), generator=g, device=DEV)
    zq = zt[:, :K] + torch.randn((B, K, V), generator=g, device=DEV)
    x = torch.randint(0, V, (B, K), generator=g, device=DEV, dtype=torch.int32)
    return (zt, zq, x, torch.rand((B, K), generator=g, device=DEV),
            torch.rand(B, generator=g, device=DEV), torch.zeros(B, device=DEV))


def test_calls_of_several_threads_on_one_stream(specv):
    sets = [_gradients(1, 3, 5000), _gradients(2, 40, 900), _gradients(4, 1100, 30)]
    inputs = _verify_inputs(40, 4, 50257)
    outs = [[torch.empty_like(t) for t in s] for s in sets]
    limits = [0.5 * float(torch.cat(s).norm()) for s in sets]
    want = []
    for s, limit, out in zip(sets, limits, outs):
        norm = float(specv.clip_grads(s, limit, out=out))
        assert abs(norm - 2 * limit) <= 1e-5 * norm
        want.append((norm, [t.clone() for t in out]))
    tokens, n = specv.verify(*inputs)
    want_tokens, want_n = tokens.clone(), n.clone()
    torch.cuda.synchronize()
    start = threading.Barrier(len(sets) + 1)
    got = [[] for _ in range(len(sets) + 1)]
    errors = []

    def work(k):
        try:
            start.wait()
            for _ in range(200):
                if k < len(sets):
                    got[k].append(specv.clip_grads(sets[k], limits[k], out=outs[k]))
                else:
                    got[k].append(specv.verify(*inputs))
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(got))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for k, (norm, out) in enumerate(want):
        assert len(got[k]) == 200 and all(float(x) == norm for x in torch.stack(got[k]).cpu())
        assert all(torch.equal(a, b) for a, b in zip(outs[k], out))
    for tokens, n in got[-1]:
        assert torch.equal(tokens, want_tokens) and torch.equal(n, want_n)


def test_scratch_released_while_another_thread_calls(specv):
    """A stream's scratch is not freed between a call's asking for it and its launches."""
    s = _gradients(2, 30, 4000)
    limit = 0.5 * float(torch.cat(s).norm())
    out = [torch.empty_like(t) for t in s]
    norm = float(specv.clip_grads(s, limit, out=out))
    got, errors = [], []

    def work():
        try:
            for _ in range(200):
                got.append(specv.clip_grads(s, limit, out=out))
        except Exception as e:
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    while t.is_alive():
        specv.release_stream()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(float(x) == norm for x in torch.stack(got).cpu())
