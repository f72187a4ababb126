"""GPU tests whose expected values leave no room for a lost or doubled entry.

Rows of equal entries: every e^{z - r} is exactly 1 and a sum of up to 2^24 of them exact
in fp32, so ln S may err by the logarithm alone.  Rows with all their mass on one entry,
for every entry of a row in turn: S is exactly 1.  And the forms of distill that only many
pairs or many chunks reach, and lists of more gradients than one launch takes.

u = 2^-24.  logf errs by 1 ulp: 2 u of the value (4 u with the roundings after it).  The
distillation kernel's log2 S is a whole exponent and the SFU's logarithm of a mantissa
near 1 (2^-22), added in fp32 (values below 32: 2^-20): the difference of two of them
times ln 2 errs by less than 2 (2^-20 + 2^-22) ln 2 < 2^-19.
"""
import math
import os

import pytest
import torch

from tests import _scoring_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = ref.U
NEG = float("-inf")


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


def _set(S):
    if S:
        os.environ["SPECV_CLUSTER_SIZE"] = str(S)
    else:
        os.environ.pop("SPECV_CLUSTER_SIZE", None)


# ------------------------------------------------------------ log probabilities
@pytest.mark.parametrize("S", [0, 1, 2, 5, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logprobs_of_equal_entries(specv, cluster_env, dtype, S):
    _set(S)
    for V in (1, 7, 255, 1000, 1024, 2047, 2049, 4096, 4097, 8193, 20011, 50257, 98304, 128256,
              300007):
        for value in (0.25, -7.0, 100.0):
            z = torch.full((3, V + 1), value, dtype=DT[dtype], device=DEV)[:, 1:]
            x = torch.tensor([0, V // 2, V - 1], dtype=torch.int32, device=DEV)
            for top in (0, 1, 20):
                got = specv.token_logprobs(z, x, top_n=top)
                ln = math.log(V)
                assert bool((got.stats[:, 0] == value).all())
                for y in (got.stats[:, 1], got.entropy, -got.logprobs):
                    assert float((y.double() - ln).abs().max()) <= 4 * U * ln, (V, value, top)
                k = min(top, V)
                if k:
                    assert torch.equal(got.top_tokens[:, :k].cpu(),
                                       torch.arange(k, dtype=torch.int32).expand(3, k))
                    assert torch.equal(got.top_logprobs[:, :k],
                                       got.logprobs.unsqueeze(-1).expand(3, k))


def _one_hot(V, at, dtype, low=-200.0):
    z = torch.full((at.numel(), V), low, dtype=DT[dtype], device=DEV)
    z[torch.arange(at.numel(), device=DEV), at] = 0.0
    return z


@pytest.mark.parametrize("V,dtype,S", [(1000, "f32", 0), (1003, "bf16", 0), (5003, "f32", 0),
                                       (9001, "bf16", 0), (5003, "bf16", 5), (9001, "f32", 16)])
def test_logprobs_of_one_entry(specv, cluster_env, V, dtype, S):
    """All the mass on one entry, for every entry of the row in turn."""
    _set(S)
    at = torch.arange(V, device=DEV)
    z = _one_hot(V, at, dtype)
    for shift in (0, 1):
        x = ((at + shift) % V).to(torch.int32)
        got = specv.token_logprobs(z, x, top_n=2)
        assert bool((got.logprobs == -200.0 * shift).all())
        assert bool((got.stats == 0).all()) and bool((got.entropy == 0).all())
        assert torch.equal(got.top_tokens[:, 0].long(), at)
        assert torch.equal(got.top_tokens[:, 1].long(), (at == 0).long())
        assert bool((got.top_logprobs[:, 0] == 0).all())
        assert bool((got.top_logprobs[:, 1] == -200).all())


# ------------------------------------------------------------------ distillation
def _divergences(specv, zt, zq, kind):
    loss, grad = specv.distill(zt, zq, kind=kind)
    only, _ = specv.distill(zt, zq, kind=kind, need_grad=False)
    return loss, only, grad


@pytest.mark.parametrize("S", [0, 1, 3, 16])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", [3, 700])
def test_distill_of_equal_entries(specv, cluster_env, dtype, S, pairs):
    """A constant target row against a draft row that is constant on a part of it."""
    _set(S)
    for V in (5, 1000, 2047, 4096, 9003, 20000, 50257, 128256):
        if V * pairs > 1 << 25:
            continue
        r = torch.arange(V, device=DEV)
        for part in (r < (V + 1) // 2, r >= V // 2, r % 3 == 1, r < V):
            zt = torch.full((1, 1, V), -2.0, dtype=DT[dtype], device=DEV).repeat(pairs, 1, 1)
            row = torch.where(part, 0.5, NEG).to(DT[dtype])
            zq = row.view(1, 1, V).repeat(pairs, 1, 1)
            H = int(part.sum())
            loss, only, grad = _divergences(specv, zt, zq, 1)
            want = math.log(V / H)
            for y in (loss, only):
                assert float((y.double() - want).abs().max()) <= 2 ** -19, (V, H)
            # q (ln q - ln p - L): each of the two differences errs as the loss does
            assert float(grad.double().abs().max()) <= 2 * 2 ** -19 / H + 1e-30
            assert bool((grad.masked_select(~part) == 0).all())
            if H < V:
                continue
            loss, only, grad = _divergences(specv, zt, zq, 0)
            assert bool((loss == 0).all()) and bool((only == 0).all()) and bool((grad == 0).all())


@pytest.mark.parametrize("V,dtype,S", [(1000, "f32", 0), (1003, "bf16", 0), (5003, "f32", 0),
                                       (9001, "bf16", 0), (4096, "f32", 0), (5003, "bf16", 5),
                                       (9001, "f32", 16)])
def test_distill_of_one_entry(specv, cluster_env, V, dtype, S):
    """All of a row's mass on one entry, for every entry of the row in turn."""
    _set(S)
    at = torch.arange(V, device=DEV)
    hot = _one_hot(V, at, dtype).unsqueeze(1)
    flat = torch.full((V, 1, V), 0.5, dtype=DT[dtype], device=DEV)
    beside = _one_hot(V, (at + 1) % V, dtype).unsqueeze(1)
    rows = torch.arange(V, device=DEV)
    for kind in (0, 1):
        # the leading row holds one entry: ln V, and 200 against an entry beside it
        t, q = (hot, flat) if kind == 0 else (flat, hot)
        loss, only, grad = _divergences(specv, t, q, kind)
        for y in (loss, only):
            assert float((y.double() - math.log(V)).abs().max()) <= 2 ** -19 + 4 * U * math.log(V)
        if kind == 0:
            want = torch.full((V, V), 1.0 / V, dtype=torch.float64, device=DEV)
            want[rows, rows] -= 1.0
            tol = 2 ** -18 / V + (ref.out_u(DT[dtype]) + 2 * U) * want.abs()
            ref.close(grad[:, 0], want, tol, "gradient")
        else:  # q (ln q - ln p - L) = 0 at the entry
            assert float(grad.double().abs().max()) <= 2 ** -18
        loss, only, grad = _divergences(specv, hot if kind == 0 else beside,
                                        beside if kind == 0 else hot, kind)
        for y in (loss, only):
            assert float((y.double() - 200.0).abs().max()) <= 8 * U * 200
        if kind == 0:
            want = torch.zeros((V, V), dtype=torch.float64, device=DEV)
            want[rows, rows] = -1.0
            want[rows, (rows + 1) % V] = 1.0
            assert float((grad[:, 0].double() - want).abs().max()) <= 2 ** -18


def _pair(shape, dtype, seed):
    B, K, V = shape
    g = torch.Generator(device=DEV).manual_seed(seed)
    zt = torch.randn((B, K + 1, V), generator=g, device=DEV) * 3.0
    zq = 0.85 * zt[:, :K] + torch.randn((B, K, V), generator=g, device=DEV)
    return zt.to(DT[dtype]), zq.to(DT[dtype])


@pytest.mark.parametrize("kind", [0, 1], ids=["forward", "reverse"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [0, 2])
@pytest.mark.parametrize("off", [0, 5], ids=["aligned", "joined"])
@pytest.mark.parametrize("chunks", [3, 4, 5, 8, 9])
def test_distill_of_many_long_pairs(specv, cluster_env, chunks, off, S, dtype, kind):
    """More CTAs than one wave: four chunks of 256 packs held, the others copied twice."""
    _set(S)
    vec = 16 // (4 if dtype == "f32" else 2)
    B, K = (350, 2) if S == 0 else (160, 2)
    V = chunks * 256 * vec * max(1, S) - off
    zt, zq = _pair((B, K, V), dtype, chunks)
    g = torch.Generator(device=DEV).manual_seed(chunks)
    w = (torch.rand((B, K), generator=g, device=DEV) + 0.5)
    w = w * (torch.rand((B, K), generator=g, device=DEV) >= 0.2)
    loss, grad = specv.distill(zt, zq, w, kind=kind)
    only, _ = specv.distill(zt, zq, w, kind=kind, need_grad=False)
    own = zq.clone()
    loss2, _ = specv.distill(zt, own, w, kind=kind, out_grad=own)
    assert torch.equal(own, grad) and torch.equal(loss, loss2)
    for b in range(0, B, 50):
        at = slice(b, b + 50)
        rl, rg, lt, gt = ref.distill(zt[at, :K], zq[at], w[at], kind == 1)
        ref.close(loss[at], rl, lt, "loss")
        ref.close(only[at], rl, lt, "loss alone")
        ref.close(grad[at], rg, gt, "gradient")


# ---------------------------------------------------------------------- clipping
CLIP_EPS = 32 * U  # as in tests/test_gpu_scoring.py


@pytest.mark.parametrize("n", [1001, 2500, 14500])
def test_clip_more_gradients_than_a_launch_takes(specv, n):
    g = torch.Generator(device=DEV).manual_seed(n)
    sizes = [(i * 37 % 251) if i % 100 else 20000 + i for i in range(n)]  # empty ones too
    flat = {t: torch.randn(sum(sizes) + 8, generator=g, device=DEV).mul_(1e-2).to(t)
            for t in DT.values()}
    at, grads, places = 3, [], []
    for i, s in enumerate(sizes):
        t = DT["bf16" if i % 3 else "f32"]
        grads.append(flat[t][at:at + s])
        places.append((t, at, s))
        at += s
    before = {t: f.clone() for t, f in flat.items()}
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in grads))
    used = {t: torch.zeros(f.numel(), dtype=torch.bool, device=DEV) for t, f in flat.items()}
    for t, a, s in places:
        used[t][a:a + s] = True
    for factor in (0.25, 2.0):
        c = min(1.0, factor * norm / (norm + 1e-6))
        into = {t: torch.full_like(f, 9.0) for t, f in flat.items()}
        got = specv.clip_grads(grads, factor * norm, out=[into[t][a:a + s] for t, a, s in places])
        assert abs(float(got) - norm) <= CLIP_EPS * norm
        for t, f in flat.items():
            assert torch.equal(f, before[t]) and bool((into[t][~used[t]] == 9.0).all())
            y = before[t][used[t]].double() * c
            ref.close(into[t][used[t]], y, (CLIP_EPS + 4 * U + ref.out_u(t)) * y.abs() + 1e-38, "out")
    # in place: as out of place
    into = {t: torch.zeros_like(f) for t, f in flat.items()}
    specv.clip_grads(grads, 0.25 * norm, out=[into[t][a:a + s] for t, a, s in places])
    got = specv.clip_grads(grads, 0.25 * norm)
    assert abs(float(got) - norm) <= CLIP_EPS * norm
    for t, f in flat.items():
        assert torch.equal(f[~used[t]], before[t][~used[t]])
        assert torch.equal(f[used[t]], into[t][used[t]])
