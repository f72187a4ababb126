"""GPU tests of sample_tokens at the ends of its range: uniforms of 0 and 1 on rows of
every length and number of threads, borders that only exact sums place, parameters of -0, the longest row.

A weight below half a unit, 2^-45 (rows of up to 2^18 entries), counts as none: at u = 0
the first kept entry that counts is drawn, at u = 1 the last.  Weights are off by up to
e = 2^-24 (4 + 4 |exponent|) of themselves, so one between 2^-45 (1 - e) and 2^-45 (1 + e)
may count or not."""
import math

import pytest
import torch

from tests import _sampling_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NEG = float("-inf")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_UNIT = 2.0 ** -45


@pytest.fixture(scope="module")
def specv():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    import speculative_decoding_verification_specv_gb300 as m
    m.load(build_if_missing=True)
    return m


def _randn(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV) * scale


def _rows(R, V, seed, dtype):
    """Rows of several kinds in turn: broad, sharp, with masked ends, with ends that weigh
    less than half a unit, with a largest entry at either end."""
    z = _randn((R, V), seed, 3.0)
    z[1::6] *= 2.0
    z[2::6, : V // 3] = NEG
    z[2::6, -(V // 5) - 1:] = NEG
    z[3::6] *= 0.1
    z[3::6, V // 2] = 32.0          # the others weigh some 2^-46
    z[4::6, : V // 2] = -60.0
    z[4::6, -(V // 9) - 1:] = -75.0
    z[5::6, 0] = 25.0
    z[5::6, V - 1] = 24.0
    return z.to(DT[dtype])


FILTERS = [dict(), dict(top_k=7), dict(top_k=40, top_p=0.9), dict(top_p=0.95), dict(top_p=0.9999),
           dict(top_k=1100, top_p=0.999), dict(top_k=3000), dict(min_p=1e-3),
           dict(top_p=0.99, min_p=1e-7)]


# a warp for each row; CTAs of 256, 512 and 1024 threads
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(12, 70), (600, 1000), (700, 5003), (200, 5003), (320, 20011),
                                 (12, 20011), (700, 50257), (6, 128256), (30, 152064)], ids=str)
def test_first_and_last(specv, R, V, dtype):
    z = _rows(R, V, V + R, dtype)
    at = torch.arange(V, device=DEV)
    for kw in FILTERS:
        for T in (1.0, 0.7):
            kept = specv.filter_logits(z, T, **kw) > NEG
            s = (z.double() - z.double().amax(-1, keepdim=True)) / T
            w, e = s.exp(), ref.U * (4 + 4 * s.clamp_min(-1e4).abs())
            must = kept & (w >= HALF_UNIT * (1 + e))
            may = kept & (w >= HALF_UNIT * (1 - e))
            del s, w, e
            for u in (0.0, 1.0):
                found = specv.sample_tokens(z, torch.full((R,), u, device=DEV), T, **kw)
                x = found.tokens.long()
                what = f"{kw} T={T} u={u}"
                assert bool(may.gather(-1, x.unsqueeze(-1)).all()), what
                if u == 0.0:
                    ok = x <= torch.where(must, at, V).amin(-1)
                    ok &= x >= torch.where(may, at, V).amin(-1)
                else:
                    ok = x >= torch.where(must, at, -1).amax(-1)
                    ok &= x <= torch.where(may, at, -1).amax(-1)
                assert bool(ok.all()), f"{what}: rows {(~ok).nonzero().view(-1)[:9].tolist()}"
                assert bool(torch.isfinite(found.logprobs).all()), what


@pytest.mark.parametrize("u", [0.36, 0.364, 0.3642], ids=str)
def test_sums_of_long_rows_of_two_levels(specv, u):
    """One row of 2^24 entries: the largest value and one of weight w, in a first half in
    pairs, then 2^20 entries of weight w, then the largest value alone.  The uniform's point
    lies among those of weight w, 14 million of the sum before and behind it: a sum that
    held entries to 2^-33 would be 50 of them off.  w is known to 2 ulp of its own (the
    exponential's): the point moves by less than 0.7 entries for the first half's 2^22
    entries of weight w and by 0.25 for those before it; the token is held to 2."""
    V, half, run = 1 << 24, 1 << 23, 1 << 20
    low = -11.7
    z = torch.zeros((1, V), device=DEV)
    z[0, :half].view(-1, 4)[:, 2:] = low
    z[0, half:half + run] = low
    unit = 2.0 ** (62 - 24)
    w = int(round(math.exp(float(torch.tensor(low))) * unit))  # rounded to a unit, not to fp32
    w32 = int(float(torch.tensor(math.exp(float(torch.tensor(low))))) * unit)
    assert abs(w - w32) <= w * ref.U
    one = int(unit)
    before = half // 2 * (one + w32)
    whole = before + run * w32 + (V - half - run) * one
    # the fp32 uniform nearest to the middle of the w's, moved by some steps
    mid = torch.tensor((before + run * w32 / 2) / whole, dtype=torch.float32)
    steps = {0.36: -3, 0.364: 0, 0.3642: 4}[u]
    point = (mid.view(torch.int32) + steps).view(torch.float32)
    t = int(float(point) * 2 ** 30) * whole >> 30
    assert float(point) * 2 ** 30 == int(float(point) * 2 ** 30)
    want = half + (t - before) // w32
    assert half < want < half + run
    found = specv.sample_tokens(z, point.view(1).to(DEV))
    assert abs(int(found.tokens[0]) - want) <= 2, int(found.tokens[0]) - want


# (the 256-thread forms with and without wider outputs too)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("R,V", [(700, 5003), (640, 20011)], ids=str)
def test_many_rows(specv, R, V, dtype, out):
    z = _randn((R, V), R + V, 3.0)
    z[::3] *= 0.2
    z = z.to(DT[dtype])
    u = torch.rand((R,), generator=torch.Generator(device=DEV).manual_seed(V), device=DEV)
    u[:20], u[20:40] = 0.0, 1.0
    for f in (dict(), dict(p=0.95), dict(k=2500), dict(a=0.05), dict(k=40, p=0.9)):
        rows = ref.Rows(z, 0.9, f.get("k", 0), f.get("p", 1.0), f.get("a", 0.0))
        kw = dict(temperature=0.9, top_k=f.get("k"), top_p=f.get("p"), min_p=f.get("a"))
        filtered = torch.full(z.shape, 7.0, dtype=DT[out], device=DEV)
        found = specv.sample_tokens(z, u, out_filtered=filtered, **kw)
        kept = rows.check_filtered(filtered, str(f))
        rows.check_draw(kept, u, found, str(f))
        alone = specv.sample_tokens(z, u, **kw)
        assert all(torch.equal(x, y) for x, y in zip(found, alone)), f
        assert torch.equal(specv.filter_logits(z, dtype=DT[out], **kw), filtered), f


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(6, 1), (12, 70), (12, 1000), (700, 5003), (12, 20011), (6, 128256)],
                         ids=str)
def test_negative_zeros_are_zeros(specv, R, V, dtype):
    """A parameter or a uniform of -0 is one of 0, as a number and in a tensor."""
    z = _rows(R, V, V, dtype) if V > 1 else torch.randn((R, 1), device=DEV).to(DT[dtype])
    u = torch.rand((R,), generator=torch.Generator(device=DEV).manual_seed(V), device=DEV)
    u[::3] = 0.0
    each = lambda x: torch.full((R,), x, device=DEV)
    some = lambda x, y: torch.where(torch.arange(R, device=DEV) % 2 == 0, x, y)
    cases = [dict(temperature=x) for x in (0.0, each(0.0), some(0.0, 0.7))]
    cases += [dict(top_p=x) for x in (0.0, each(0.0), some(0.0, 0.9))]
    cases += [dict(top_p=0.0, top_k=k) for k in (20, 3000)]
    cases += [dict(temperature=0.0, top_k=50, top_p=0.0, min_p=0.0), dict(min_p=some(0.0, 0.1)), dict()]

    def negated(x):
        if isinstance(x, torch.Tensor):
            return torch.where(x == 0, -0.0, x)
        return -0.0 if isinstance(x, float) and x == 0 else x

    for kw in cases:
        neg = {k: negated(x) for k, x in kw.items()}
        for v in neg.values():  # (there is something to test)
            if isinstance(v, torch.Tensor):
                assert bool((torch.signbit(v) & (v == 0)).any())
        out, want = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
        a = specv.sample_tokens(z, u, out_filtered=want, **kw)
        b = specv.sample_tokens(z, negated(u), out_filtered=out, **neg)
        torch.cuda.synchronize()
        assert bool((a.tokens >= 0).all())
        assert all(torch.equal(x, y) for x, y in zip(a, b)), kw
        assert torch.equal(out, want) and torch.equal(specv.filter_logits(z, **neg), want), kw
        if V > 1 and not isinstance(kw.get("temperature", 1), torch.Tensor) and kw.get("temperature") == 0.0:
            first = torch.where(z == z.amax(-1, keepdim=True), torch.arange(V, device=DEV), V).amin(-1)
            assert torch.equal(b.tokens.long(), first)


def test_the_longest_row(specv):
    """2^31 - 1 entries, 18, 20 and 19 among entries of -20: those weigh 2^-57, below half a
    unit (2^-31 here), and count as none in the sums; the three hold 0.09, 0.665 and 0.245 of
    the whole."""
    V = (1 << 31) - 1
    at = [5, (1 << 30) + 1, V - 2]
    z = torch.full((1, V), -20.0, dtype=torch.bfloat16, device=DEV)
    z[0, at] = torch.tensor([18.0, 20.0, 19.0], dtype=torch.bfloat16, device=DEV)
    share = torch.softmax(torch.tensor([18.0, 20.0, 19.0], dtype=torch.float64), 0)
    out = torch.empty_like(z)
    for kw, kept in ((dict(), [0, 1, 2]), (dict(top_k=2), [1, 2]), (dict(top_p=0.5), [1]),
                     (dict(top_p=0.9), [1, 2]), (dict(min_p=0.2), [1, 2]), (dict(temperature=0.0), [1]),
                     (dict(top_k=100000), [0, 1, 2]), (dict(top_k=100000, top_p=0.9), [1, 2])):
        p = share[kept] / share[kept].sum()
        upto = p.cumsum(0)
        filtered = specv.filter_logits(z, out=out, **kw)
        some = int((filtered > NEG).sum())
        if kw == dict():
            assert some == V
        elif kw == dict(top_k=100000):  # the three and the first others, in index order
            assert some == 100000 and bool((filtered[0, : 100000 - 2] > NEG).all())
        else:
            assert some == len(kept)
        for j in kept:
            assert float(filtered[0, at[j]]) == (0.0 if "temperature" in kw else float(z[0, at[j]]))
        for u, j in ((0.0, 0), (0.5, int((upto <= 0.5).sum())), (1.0, len(kept) - 1)):
            found = specv.sample_tokens(z, torch.full((1,), u, device=DEV), **kw)
            assert int(found.tokens[0]) == at[kept[j]], (kw, u)
            # (the sum of a row that nothing filters is in fp32, off by some hundred roundings)
            assert abs(float(found.logprobs[0]) - math.log(p[j])) <= 1e-4, (kw, u)
