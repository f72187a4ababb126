"""The C-ABI boundary of the operators on the step's logits without a GPU: bad
arguments are rejected on the host and launch nothing."""
import ctypes

import pytest

import speculative_decoding_verification_specv_gb300 as specv

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module", autouse=True)
def lib():
    return specv.load(build_if_missing=True)


def _logprobs(B=2, N=3, V=100, sb=300, sn=100, dtype=0, top=2, null=None, at=None):
    p = [FAKE] * 7
    if null is not None:
        p[null] = None
    if at is not None:
        p[0] = at
    return specv.raw_call("specv_token_logprobs", p[0], p[1], B, N, V, sb, sn, dtype, top, p[2],
                          p[3], p[4], p[5], p[6], None)


@pytest.mark.parametrize("kw", [*(dict(null=i) for i in range(7)), dict(B=0), dict(N=0), dict(V=0),
                                dict(B=-1), dict(sb=-1), dict(sn=-1), dict(dtype=2), dict(dtype=-1),
                                dict(top=33), dict(top=-1), dict(B=1 << 30, N=2),
                                dict(B=1 << 20, sb=1 << 50), dict(at=FAKE + 2),
                                dict(at=FAKE + 1, dtype=1)], ids=str)
def test_token_logprobs_validates(kw):
    assert _logprobs(**kw) == 1


def test_token_logprobs_checks_alignment():
    for i in range(7):  # every array at 2 bytes off, the statistics also at 4
        for off in (2, 4) if i == 4 else (2,):
            p = [FAKE] * 7
            p[i] += off
            assert specv.raw_call("specv_token_logprobs", p[0], p[1], 2, 3, 100, 300, 100, 0, 2,
                                  p[2], p[3], p[4], p[5], p[6], None) == 1, (i, off)
    for i in range(7):
        for off in (2, 4) if i == 2 else (2,):
            p = [FAKE] * 7
            p[i] += off
            assert specv.raw_call("specv_token_logprobs_backward", *p[:6], 2, 3, 100, 300, 100, 0,
                                  p[6], None) == 1, (i, off)
    for i in range(5):
        p = [FAKE] * 5
        p[i] += 2
        assert specv.raw_call("specv_distill", p[0], p[1], p[2], 2, 3, 100, 400, 100, 300, 100, 0,
                              0, p[3], p[4], None) == 1, i


def _backward(B=2, N=3, V=100, sb=300, sn=100, dtype=0, null=None, out=FAKE):
    p = [FAKE] * 5
    if null is not None:
        p[null] = None
    return specv.raw_call("specv_token_logprobs_backward", p[0], p[1], p[2], p[3], p[4], None, B, N,
                          V, sb, sn, dtype, out, None)


@pytest.mark.parametrize("kw", [*(dict(null=i) for i in range(5)), dict(out=None), dict(B=0),
                                dict(N=-2), dict(V=0), dict(sb=-5), dict(dtype=7),
                                dict(out=FAKE + 2), dict(B=1 << 31)], ids=str)
def test_token_logprobs_backward_validates(kw):
    assert _backward(**kw) == 1


def _distill(B=2, K=3, V=100, t=(400, 100), d=(300, 100), dtype=0, kind=0, null=None, grad=FAKE,
             target=FAKE):
    p = [target, FAKE, FAKE]
    if null is not None:
        p[null] = None
    return specv.raw_call("specv_distill", p[0], p[1], FAKE, B, K, V, *t, *d, dtype, kind, p[2],
                          grad, None)


@pytest.mark.parametrize("kw", [*(dict(null=i) for i in range(3)), dict(B=0), dict(K=0), dict(V=-1),
                                dict(t=(-1, 0)), dict(d=(0, -1)), dict(dtype=2), dict(kind=2),
                                dict(kind=-1), dict(grad=FAKE + 1), dict(target=FAKE + 2),
                                dict(B=1 << 16, K=1 << 15)], ids=str)
def test_distill_validates(kw):
    assert _distill(**kw) == 1


def _clip(entries, n=None, max_norm=1.0, norm=FAKE, null=False):
    flat = [v for e in entries for v in e]
    table = (ctypes.c_int64 * len(flat))(*flat)
    return specv.raw_call("specv_clip_grads", None if null else table,
                          len(entries) if n is None else n, max_norm, norm, None)


def test_clip_grads_validates():
    good = (FAKE, FAKE, 10, 0)
    assert _clip([good], max_norm=-1.0) == 1
    assert _clip([good], max_norm=float("nan")) == 1
    assert _clip([good], norm=None) == 1
    assert _clip([good], n=-1) == 1
    assert _clip([good], norm=FAKE + 2) == 1
    assert _clip([good], null=True) == 1
    for bad in ((0, FAKE, 10, 0), (FAKE, 0, 10, 0), (FAKE, FAKE, -1, 0), (FAKE, FAKE, 10, 2),
                (FAKE + 2, FAKE, 10, 0), (FAKE, FAKE + 1, 10, 1), (FAKE, FAKE, 1 << 61, 0)):
        assert _clip([good, bad]) == 1, bad


def test_binding_refuses_host_tensors():
    import torch
    z, x = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: specv.token_logprobs(z, x), lambda: specv.distill(z, z),
                 lambda: specv.clip_grads([z], 1.0)):
        with pytest.raises(ValueError):
            call()
