"""GPU tests of distill on pairs whose finite logits lie far apart: masks of -2e4,
-65504, -1e9 and the type's lowest value in one row of a pair or differing in both, as
runs (whole lanes, chunks and CTAs see nothing else) and spread, in every kernel form.

The tolerances, with u = 2^-24, a the leading row's log probabilities, c the other's, da
and dc the distances of the logits from their rows' maxima:
* a term e^a errs relatively by the two roundings of its exponent's argument (2 u |da|,
  doubled for a reference that is not the maximum), the exponential's 2 ulp and those of
  up to eight moves of the reference: eps = u (64 + 4 |da|);
* a sum by n u with n additions one after the other: rows of up to 2048 entries take 64 in
  a lane, longer ones V / 128 in a thread, 64 further ones merge: n = V / 128 + 128;
* a difference of logits by u times the two distances from the references and itself:
  3 u (|da| + |dc| + 32).
The divergence is T / S_a - ln S_a + ln S_c, the logarithms within 8 u of their size.
"""
import os

import pytest
import torch

from tests import _scoring_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def specv():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    import speculative_decoding_verification_specv_gb300 as m
    m.load(build_if_missing=True)
    return m


@pytest.fixture
def cluster_env():
    old = os.environ.get("SPECV_CLUSTER_SIZE")
    yield
    if old is None:
        os.environ.pop("SPECV_CLUSTER_SIZE", None)
    else:
        os.environ["SPECV_CLUSTER_SIZE"] = old


def _randn(shape, seed, scale):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV) * scale


def far_ref(target, draft, w, reverse):
    """(loss, gradient, loss tolerance, gradient tolerance) in 64 bits; every logit finite."""
    u = ref.U
    t, q = target.double(), draft.double()
    V = q.shape[-1]
    lt, lq = torch.log_softmax(t, -1), torch.log_softmax(q, -1)
    dt, dq = t - t.amax(-1, keepdim=True), q - q.amax(-1, keepdim=True)
    st, sq = dt.exp().sum(-1).log(), dq.exp().sum(-1).log()
    (a, c, da, dc) = (lq, lt, dq.abs(), dt.abs()) if reverse else (lt, lq, dt.abs(), dq.abs())
    lead, diff = a.exp(), a - c
    kl = (lead * diff).sum(-1)
    n = V / 128 + 128
    eps = u * (64 + 4 * da)
    sum_a = n * u + (lead * eps).sum(-1)
    sum_c = n * u + (c.exp() * u * (64 + 4 * dc)).sum(-1)
    kl_tol = ((lead * diff.abs() * (n * u + eps)).sum(-1) + 3 * u * (lead * (da + dc + 32)).sum(-1)
              + (kl.abs() + st + sq + 32) * (sum_a + 4 * u) + sum_a + sum_c + 8 * u * (1 + st + sq))
    wx, k = w.double().unsqueeze(-1), kl.unsqueeze(-1)
    if reverse:
        grad = wx * lead * (diff - k)
        tol = lead * ((eps + sum_a.unsqueeze(-1) + 8 * u) * (diff.abs() + k.abs())
                      + 4 * u * (da + dc + k.abs() + (st + sq).unsqueeze(-1) + 32)
                      + kl_tol.unsqueeze(-1))
    else:
        p, eq = a.exp(), c.exp()
        grad = wx * (eq - p)
        tol = (p * (eps + sum_a.unsqueeze(-1)) + eq * (u * (64 + 4 * dc) + sum_c.unsqueeze(-1)))
    tol = wx.abs() * tol + ref.out_u(draft.dtype) * grad.abs() + 1e-36
    return w * kl, grad, w.abs() * kl_tol + 2 * u * (w * kl).abs(), tol


def _pairs(V, dtype):
    """[P][1][V] target and draft rows."""
    r = torch.arange(V, device=DEV)
    t, q = _randn((V,), V, 3.0), _randn((V,), V + 1, 3.0)
    vec = 16 // (4 if dtype == "f32" else 2)
    places = [r >= V // 2, r < V // 3, r % 7 == 3, (r // vec) % 32 == 5, r == V - 1]
    rows = []
    for fill in (-2e4, -65504.0, -1e9, torch.finfo(DT[dtype]).min):
        for m in places:
            rows += [(t, q.masked_fill(m, fill)), (t.masked_fill(m, fill), q)]
    tail, head = places[0], places[1]
    low = torch.finfo(DT[dtype]).min
    ramp = r * (-3e4 / V)
    rows += [(t.masked_fill(tail, -1e9), q.masked_fill(tail, low)),
             (t.masked_fill(tail, low), q.masked_fill(tail, -65504.0)),
             (t.masked_fill(head, -1e5), q.masked_fill(tail, -1e9)),
             (t.masked_fill(tail, low), q.masked_fill(head, low)),
             (t, ramp), (ramp, q), (ramp, ramp.flip(0)), (t + 3e4, q - 3e4)]
    return (torch.stack([a for a, _ in rows]).to(DT[dtype]).unsqueeze(1),
            torch.stack([b for _, b in rows]).to(DT[dtype]).unsqueeze(1))


def _check(specv, zt, zq, kind, copies=1):
    P = zq.shape[0]
    w = (torch.rand((P, 1), generator=torch.Generator(device=DEV).manual_seed(P), device=DEV) + 0.25)
    rl, rg, lt, gt = far_ref(zt, zq, w, kind == 1)
    many = [x.repeat(copies, *[1] * (x.dim() - 1)) for x in (zt, zq, w)]
    loss, grad = specv.distill(*many, kind=kind)
    only, _ = specv.distill(*many, kind=kind, need_grad=False)
    for k in sorted({0, copies // 2, copies - 1}):
        at = slice(k * P, (k + 1) * P)
        ref.close(loss[at], rl, lt, "loss")
        ref.close(only[at], rl, lt, "loss alone")
        ref.close(grad[at], rg, gt, "gradient")


@pytest.mark.parametrize("kind", [0, 1], ids=["forward", "reverse"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 33, 128, 512, 1000, 2047, 9003, 40960, 128256])
def test_distill_far_logits(specv, V, dtype, kind):
    _check(specv, *_pairs(V, dtype), kind)


@pytest.mark.parametrize("S", [1, 3, 16])
@pytest.mark.parametrize("V,dtype", [(9003, "f32"), (40960, "bf16"), (2500, "f32"), (700, "bf16")])
def test_distill_far_logits_in_clusters(specv, cluster_env, V, dtype, S):
    os.environ["SPECV_CLUSTER_SIZE"] = str(S)
    for kind in (0, 1):
        _check(specv, *_pairs(V, dtype), kind)


@pytest.mark.parametrize("V,dtype", [(9003, "f32"), (9216, "f32"), (12000, "bf16"), (17003, "bf16"),
                                     (500, "f32")])
def test_distill_far_logits_of_many_pairs(specv, V, dtype):
    """More pairs than one wave of CTAs holds."""
    for kind in (0, 1):
        _check(specv, *_pairs(V, dtype), kind, copies=30)
