"""GPU tests of token_logprobs, token_logprobs_backward, distill and clip_grads
against 64-bit restatements (tests/_scoring_ref.py, which derives the tolerances):
lengths from one entry to long rows, odd vocabularies, strides, both types, masked
and empty rows, NaN and infinities, ties, left-out rows, other streams, graphs."""
import math
import os

import pytest
import torch

from tests import _scoring_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NEG = float("-inf")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LOWEST = {k: torch.finfo(v).min for k, v in DT.items()}


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


def _randn(shape, seed, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV) * scale


def _tokens(shape, V, seed, skip=0.0):
    g = torch.Generator(device=DEV).manual_seed(1000 + seed)
    x = torch.randint(0, V, shape, generator=g, device=DEV, dtype=torch.int32)
    drop = torch.rand(shape, generator=g, device=DEV) < skip
    return torch.where(drop, torch.full_like(x, -1), x)


def _check_logprobs(specv, logits, tokens, top_n):
    got = specv.token_logprobs(logits, tokens, top_n=top_n)
    torch.cuda.synchronize()
    lp, H, M, ln, tt, tl, tol = ref.token_logprobs(logits, tokens, top_n)
    ref.close(got.logprobs.cpu(), lp, tol + 4 * ref.U * lp.abs().nan_to_num(0, 0, 0), "logprobs")
    ref.close(got.entropy.cpu(), H, 2 * tol, "entropy")
    ref.close(got.stats[..., 0].cpu(), M, torch.zeros_like(M), "maximum")
    ref.close(got.stats[..., 1].cpu(), ln, tol, "ln sum")
    if top_n:
        assert torch.equal(got.top_tokens.cpu(), tt)
        t = tol.unsqueeze(-1) + 4 * ref.U * tl.abs().nan_to_num(0, 0, 0)
        ref.close(got.top_logprobs.cpu(), tl, t, "top logprobs")
    else:
        assert got.top_tokens is None and got.top_logprobs is None
    return got


# ------------------------------------------------------------ log probabilities
SHAPES = [(1, 1, 1), (1, 1, 2), (3, 2, 7), (1, 4, 31), (5, 3, 32), (2, 3, 33), (7, 1, 255),
          (2, 2, 1000), (3, 2, 1001), (2, 2, 2047), (1, 3, 2049), (4, 3, 4100), (2, 2, 20011),
          (1, 9, 50257), (2, 3, 128256), (1, 2, 300007)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_logprobs_shapes(specv, shape, dtype):
    B, N, V = shape
    z = _randn(shape, V).to(DT[dtype])
    for top in (0, 5, 32):
        _check_logprobs(specv, z, _tokens((B, N), V, V, skip=0.2), top)


@pytest.mark.parametrize("S", [1, 2, 3, 8, 16])
def test_logprobs_cluster_sizes(specv, cluster_env, S):
    os.environ["SPECV_CLUSTER_SIZE"] = str(S)
    for V, dtype in ((40001, "bf16"), (9001, "f32"), (65536, "f32"), (5000, "bf16")):
        _check_logprobs(specv, _randn((2, 2, V), S).to(DT[dtype]), _tokens((2, 2), V, S), 20)


def _special_rows(V, dtype):
    """Rows that break a careless softmax or selection, by name."""
    low = LOWEST[dtype]
    r = torch.arange(V, device=DEV, dtype=torch.float32)
    z = _randn((V,), 5)
    rows = {}
    rows["empty"] = torch.full((V,), NEG, device=DEV)
    one = rows["empty"].clone()
    one[V // 2] = -3.0
    rows["one entry"] = one
    few = rows["empty"].clone()
    few[:: max(1, V // 3)] = 1.5
    rows["few entries"] = few
    rows["all lowest"] = torch.full((V,), low, device=DEV)
    lm = torch.full((V,), low, device=DEV)
    lm[V // 3: V // 3 + 4] = z[:4] if V >= 12 else z[:lm[V // 3: V // 3 + 4].numel()]
    rows["lowest masks"] = lm
    lowinf = torch.full((V,), NEG, device=DEV)
    lowinf[V - 1] = low
    rows["lowest among masks"] = lowinf
    rows["masked prefix"] = torch.where(r < (2 * V) // 3, torch.full_like(z, NEG), z)
    rows["masked tail"] = torch.where(r >= V // 3 + 1, torch.full_like(z, NEG), z)
    rows["masked every other"] = torch.where(r % 2 == 1, torch.full_like(z, NEG), z)
    rows["constant"] = torch.full((V,), 0.25, device=DEV)
    rows["zeros of both signs"] = torch.where(r % 3 == 0, -0.0, 0.0)
    rows["ascending"] = r * 1e-3
    rows["descending"] = -r * 1e-3
    rows["a few levels"] = (r * 7 % 5).floor()
    rows["peaked"] = torch.where(r == V - 1, torch.full_like(z, 60.0), z)
    rows["large"] = z * 30 + 3000.0
    rows["small"] = z * 30 - 3000.0
    big = torch.where(r % 256 == 3, 50.0 + r * 1e-3, z)  # many of the largest in one place
    rows["periodic"] = big
    rows["periodic long"] = torch.where(r % 2048 < 8, 50.0 + r * 1e-4, z)
    nan = z.clone()
    nan[V // 2] = float("nan")
    rows["nan"] = nan
    inf = z.clone()
    inf[V // 3] = math.inf
    rows["inf"] = inf
    mixed = torch.full((V,), NEG, device=DEV)
    mixed[0] = float("nan")
    rows["nan among masks"] = mixed
    rows["all nan"] = torch.full((V,), float("nan"), device=DEV)
    return rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 5, 32, 257, 1000, 2500, 8200, 40003])
def test_logprobs_special_rows(specv, V, dtype):
    rows = _special_rows(V, dtype)
    z = torch.stack(list(rows.values())).to(DT[dtype])
    x = torch.full((z.shape[0],), V // 2, dtype=torch.int32, device=DEV)
    for top in (1, 5, 20, 32):
        _check_logprobs(specv, z, x, top)
    x = torch.zeros_like(x)
    _check_logprobs(specv, z, x, 3)


@pytest.mark.parametrize("S", [2, 5, 16])
def test_logprobs_special_rows_in_clusters(specv, cluster_env, S):
    os.environ["SPECV_CLUSTER_SIZE"] = str(S)
    for V, dtype in ((9003, "f32"), (40960, "bf16")):
        z = torch.stack(list(_special_rows(V, dtype).values())).to(DT[dtype])
        x = torch.full((z.shape[0],), V - 1, dtype=torch.int32, device=DEV)
        for top in (1, 20, 32):
            _check_logprobs(specv, z, x, top)


@pytest.mark.parametrize("dtype,period,width", [("bf16", 2048, 8), ("f32", 1024, 4)])
def test_logprobs_crowded_rows(specv, cluster_env, dtype, period, width):
    """Rows whose largest entries all fall to one thread of the streaming loop: more of
    them than the selection collects, so that the repeated search decides."""
    os.environ["SPECV_CLUSTER_SIZE"] = "1"
    V = 160001
    r = torch.arange(V, device=DEV, dtype=torch.float32)
    z = _randn((V,), 7)
    big = r % period < width
    rows = [torch.where(big, 40.0 + (r * 13 % 61) * 0.25, z),   # with many ties
            torch.where(big, 40.0 + r * 1e-4, z),               # rising
            torch.where(big, 90.0 - r * 1e-4, z),               # falling
            torch.where(big, z.abs() + 30.0, z).masked_fill(r % 3 == 1, NEG)]
    z = torch.stack(rows).to(DT[dtype])
    x = torch.full((len(rows),), 5, dtype=torch.int32, device=DEV)
    for top in (1, 20, 32):
        _check_logprobs(specv, z, x, top)


def test_logprobs_invalid_and_absent_tokens(specv):
    for V in (40, 3001, 50000):
        z = _randn((2, 5, V), 3)
        x = torch.tensor([[-1, 0, V, -2, V - 1], [2 ** 31 - 1, -2 ** 31, -1, 1, 2]],
                         dtype=torch.int32, device=DEV)
        z[0, 0] = float("nan")  # a row without a token is not looked at
        _check_logprobs(specv, z, x, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [70, 1024, 5003, 33000])
def test_logprobs_strided_views(specv, dtype, V):
    full = _randn((3, 6, V + 13), 4).to(DT[dtype])
    padded = full[..., :V]                      # a padded vocabulary
    shifted = full[:, :5, 1:V + 1]              # rows from an odd offset, fewer positions
    turned = full[..., :V].transpose(0, 1)      # the leading dimensions in the other order
    shared = full[:1, :, 3:V + 3].expand(4, 6, V)
    for z in (padded, shifted, turned, shared, full[1, :, :V], full[:, 2:3, 5:V + 5]):
        x = _tokens(z.shape[:-1], V, V, skip=0.1)
        got = _check_logprobs(specv, z, x, 7)
        g, h = _randn(x.shape, 8, 1.0), _randn(x.shape, 9, 0.3)
        grad = specv.token_logprobs_backward(z, x, got.stats, got.entropy, g, h)
        want, tol = ref.logprobs_gradient(z, x, g, h)
        assert grad.is_contiguous() and grad.dtype == z.dtype
        ref.close(grad, want, tol, "gradient")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_logprobs_gradient(specv, shape, dtype):
    B, N, V = shape
    z = _randn(shape, V + 1).to(DT[dtype])
    x = _tokens((B, N), V, V, skip=0.2)
    fwd = specv.token_logprobs(z, x)
    g, h = _randn((B, N), 8, 1.0), _randn((B, N), 9, 0.3)
    for hh in (h, None):
        grad = specv.token_logprobs_backward(z, x, fwd.stats, fwd.entropy, g, hh)
        want, tol = ref.logprobs_gradient(z, x, g, torch.zeros_like(g) if hh is None else hh)
        ref.close(grad, want, tol, "gradient")
    # in place
    own = z.clone()
    same = specv.token_logprobs_backward(own, x, fwd.stats, fwd.entropy, g, None, out=own)
    assert same is own and torch.equal(own, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 33, 1000, 8200])
def test_logprobs_gradient_special_rows(specv, V, dtype):
    z = torch.stack(list(_special_rows(V, dtype).values())).to(DT[dtype])
    for at in (0, V // 2, V - 1):
        x = torch.full((z.shape[0],), at, dtype=torch.int32, device=DEV)
        fwd = specv.token_logprobs(z, x)
        g, h = _randn(x.shape, 8, 1.0), _randn(x.shape, 9, 0.3)
        grad = specv.token_logprobs_backward(z, x, fwd.stats, fwd.entropy, g, h)
        want, tol = ref.logprobs_gradient(z, x, g, h)
        ref.close(grad, want, tol, "gradient")
    x = torch.tensor([-1, -2, V, 0], dtype=torch.int32, device=DEV)
    z = _randn((4, V), 2).to(DT[dtype])
    fwd = specv.token_logprobs(z, x)
    grad = specv.token_logprobs_backward(z, x, fwd.stats, fwd.entropy, _randn((4,), 1), None)
    assert bool((grad[0] == 0).all()) and bool(torch.isnan(grad[1:3]).all())
    assert bool(torch.isfinite(grad[3]).all())


def test_logprobs_gradient_against_differences(specv):
    """The directional derivative of the 64-bit value along random directions."""
    V = 777
    z = _randn((4, V), 11, 2.0)
    x = _tokens((4,), V, 3)
    g, h = _randn((4,), 12, 1.0), _randn((4,), 13, 1.0)
    fwd = specv.token_logprobs(z, x)
    grad = specv.token_logprobs_backward(z, x, fwd.stats, fwd.entropy, g, h).double()

    def value(y):
        lp = torch.log_softmax(y, -1)
        H = -(lp.exp() * lp).sum(-1)
        return (g.double() * lp.gather(-1, x.long().unsqueeze(-1)).squeeze(-1) + h.double() * H).sum()

    for seed in range(4):
        d = _randn((4, V), 20 + seed, 1.0).double()
        s = 1e-5
        slope = (value(z.double() + s * d) - value(z.double() - s * d)) / (2 * s)
        # truncation s^2 |f'''| / 6 and cancellation 1e-16 |f| / s are below 1e-9; the
        # kernel's entries err by their tolerance, against |d| <= 6
        _, tol = ref.logprobs_gradient(z, x, g, h)
        assert abs(float(slope - (grad * d).sum())) <= 6 * float(tol.sum()) + 1e-8


# ------------------------------------------------------------------ distillation
def _check_distill(specv, zt, zq, weight, kind, **kw):
    loss, grad = specv.distill(zt, zq, weight, kind=kind, **kw)
    torch.cuda.synchronize()
    B, K, V = zq.shape
    w = torch.ones((B, K), device=DEV) if weight is None else weight
    rl, rg, lt, gt = ref.distill(zt[:, :K], zq, w, kind == 1)
    ref.close(loss, rl, lt, "loss")
    assert grad.is_contiguous() and grad.dtype == zq.dtype and grad.shape == zq.shape
    ref.close(grad, rg, gt, "gradient")
    only, none = specv.distill(zt, zq, weight, kind=kind, need_grad=False)
    assert none is None
    ref.close(only, rl, lt, "loss alone")
    return loss, grad


def _pair(shape, dtype, seed, noise=1.0):
    B, K, V = shape
    zt = _randn((B, K + 1, V), seed)
    zq = 0.85 * zt[:, :K] + _randn((B, K, V), seed + 1, noise)
    return zt.to(DT[dtype]), zq.to(DT[dtype])


def _weights(shape, seed, skip):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.rand(shape, generator=g, device=DEV) + 0.5
    return w * (torch.rand(shape, generator=g, device=DEV) >= skip)


@pytest.mark.parametrize("kind", [0, 1], ids=["forward", "reverse"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_distill_shapes(specv, shape, dtype, kind):
    B, K, V = shape
    zt, zq = _pair(shape, dtype, V)
    _check_distill(specv, zt, zq, _weights((B, K), V, 0.25), kind)
    _check_distill(specv, zt[:, :K], zq, None, kind)


@pytest.mark.parametrize("S", [1, 2, 3, 8, 16])
def test_distill_cluster_sizes(specv, cluster_env, S):
    os.environ["SPECV_CLUSTER_SIZE"] = str(S)
    for V, dtype in ((40001, "bf16"), (9001, "f32"), (65536, "f32"), (5000, "bf16"),
                     (270336, "bf16")):
        zt, zq = _pair((2, 2, V), dtype, S)
        for kind in (0, 1):
            _check_distill(specv, zt, zq, _weights((2, 2), S, 0.2), kind)


def _special_pairs(V, dtype):
    low = LOWEST[dtype]
    r = torch.arange(V, device=DEV, dtype=torch.float32)
    t, q = _randn((V,), 5), _randn((V,), 6)
    empty = torch.full((V,), NEG, device=DEV)
    tail = r >= V // 2 + 1
    odd = r % 2 == 1
    nan = t.clone()
    nan[V // 2] = float("nan")
    inf = t.clone()
    inf[V // 2] = math.inf
    one = empty.clone()
    one[V // 3] = 2.0
    pairs = [
        (empty, q), (t, empty), (empty, empty),                     # nothing left
        (t.masked_fill(tail, NEG), q.masked_fill(tail, NEG)),       # both padded
        (t.masked_fill(odd, NEG), q.masked_fill(odd, NEG)),
        (t.masked_fill(tail, NEG), q),                              # p = 0 where q > 0
        (t, q.masked_fill(tail, NEG)),                              # q = 0 where p > 0
        (t.masked_fill(tail, low), q.masked_fill(tail, low)),       # masks of the lowest value
        (t.masked_fill(tail, NEG), q.masked_fill(tail, low)),
        (torch.full((V,), low, device=DEV), torch.full((V,), low, device=DEV)),
        (one, one), (one, q), (t, one),
        (t, t), (t * 0, q * 0), (t * 30 + 3000, q + 3000), (t - 3000, q * 3 - 3000),
        (nan, q), (t, nan), (inf, q), (t, inf), (nan, empty), (empty, inf),
    ]
    return (torch.stack([a for a, _ in pairs]).to(DT[dtype]).unsqueeze(1),
            torch.stack([b for _, b in pairs]).to(DT[dtype]).unsqueeze(1))


@pytest.mark.parametrize("kind", [0, 1], ids=["forward", "reverse"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 5, 33, 1000, 2500, 40003])
def test_distill_special_rows(specv, V, dtype, kind):
    zt, zq = _special_pairs(V, dtype)
    _check_distill(specv, zt, zq, None, kind)


@pytest.mark.parametrize("S", [2, 16])
def test_distill_special_rows_in_clusters(specv, cluster_env, S):
    os.environ["SPECV_CLUSTER_SIZE"] = str(S)
    for V, dtype in ((9003, "f32"), (40960, "bf16")):
        zt, zq = _special_pairs(V, dtype)
        for kind in (0, 1):
            _check_distill(specv, zt, zq, None, kind)


def test_distill_identical_rows_and_odd_weights(specv):
    for V, dtype in ((1000, "f32"), (50001, "bf16"), (128256, "f32")):
        zt, _ = _pair((2, 3, V), dtype, 3)
        zq = zt[:, :3].contiguous()
        for kind in (0, 1):
            loss, grad = specv.distill(zt, zq, kind=kind)
            assert float(loss.abs().max()) <= 1e-6 and float(grad.abs().float().max()) <= 1e-6
        w = torch.tensor([[0.0, float("nan"), -2.0], [1e-30, 0.0, 3e4]], device=DEV)
        zt[0, 0, 5] = float("nan")  # a position of weight 0 is not read
        loss, grad = specv.distill(zt, zq * 0.5, w)
        assert loss[0, 0] == 0 and loss[1, 1] == 0 and torch.isnan(loss[0, 1]) and loss[0, 2] <= 0
        assert bool((grad[0, 0] == 0).all()) and bool((grad[1, 1] == 0).all())
        assert bool(torch.isnan(grad[0, 1]).all()) and bool(torch.isfinite(grad[1, 2]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [70, 1024, 5003, 33000])
def test_distill_strided_views_and_in_place(specv, dtype, V):
    ft, fq = _randn((3, 6, V + 13), 4).to(DT[dtype]), _randn((3, 6, V + 13), 5).to(DT[dtype])
    w = _weights((3, 5), 3, 0.2)
    for zt, zq in ((ft[..., :V], fq[:, :5, :V]), (ft[:, :5, 1:V + 1], fq[:, :5, 2:V + 2]),
                   (ft[:, 1:, 3:V + 3], fq[:, :5, 3:V + 3]),
                   (ft[:1, :, :V].expand(3, 6, V), fq[:1, :5, :V].expand(3, 5, V))):
        for kind in (0, 1):
            _check_distill(specv, zt, zq, w, kind)
    zq = fq[:, :5, :V].contiguous()
    for kind in (0, 1):
        loss, grad = specv.distill(ft[..., :V], zq, w, kind=kind)
        own = zq.clone()
        loss2, same = specv.distill(ft[..., :V], own, w, kind=kind, out_grad=own)
        assert same is own and torch.equal(own, grad) and torch.equal(loss, loss2)


@pytest.mark.parametrize("kind", [0, 1], ids=["forward", "reverse"])
def test_distill_gradient_against_differences(specv, kind):
    zt, zq = _pair((2, 2, 777), "f32", 31)
    w = _weights((2, 2), 5, 0.0)
    _, grad = specv.distill(zt, zq, w, kind=kind)

    def value(y):
        lt, lq = torch.log_softmax(zt[:, :2].double(), -1), torch.log_softmax(y, -1)
        a, c = (lq, lt) if kind else (lt, lq)
        return (w.double() * (a.exp() * (a - c)).sum(-1)).sum()

    _, _, _, tol = ref.distill(zt[:, :2], zq, w, kind == 1)
    for seed in range(4):
        d = _randn(zq.shape, 40 + seed, 1.0).double()
        s = 1e-5
        slope = (value(zq.double() + s * d) - value(zq.double() - s * d)) / (2 * s)
        assert abs(float(slope - (grad.double() * d).sum())) <= 6 * float(tol.sum()) + 1e-8


# ---------------------------------------------------------------------- clipping
def _norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


# 8192 squares in fp32 (32 additions per thread and the merge's 0 in fp32): 40 u of the
# sum, half of it for the root, and the roundings of the root and the factor
CLIP_EPS = 32 * ref.U


def _check_clip(specv, grads, max_norm, out=None):
    before = [g.clone() for g in grads]
    norm = specv.clip_grads(grads, max_norm, out=out)
    torch.cuda.synchronize()
    want = _norm(before)
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= CLIP_EPS * want + 1e-30
    c = min(1.0, max_norm / (want + 1e-6))
    for g, b, o in zip(grads, before, grads if out is None else out):
        if out is not None and o is not g:
            assert torch.equal(g, b)
        y = b.double() * c
        # the factor is 1 or not within its own rounding of the limit
        tol = (CLIP_EPS + 4 * ref.U + ref.out_u(b.dtype)) * y.abs() + 1e-38
        ref.close(o.reshape(b.shape), y, tol, "clipped")
    return norm


def _grads(sizes, seed, scale=1e-2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(n, generator=g, device=DEV).mul_(scale).to(DT["bf16" if i % 3 else "f32"])
            for i, n in enumerate(sizes)]


@pytest.mark.parametrize("sizes", [(1,), (0, 1, 0), (5, 17, 255), (8191, 8192, 8193), (100003,),
                                   (1 << 20, 3, 70001, 0, 12), tuple(range(1, 420)),
                                   tuple(i * 97 % 9001 for i in range(900))],
                         ids=lambda s: f"n{len(s)}sum{sum(s)}")
def test_clip_sizes(specv, sizes):
    for factor in (0.3, 1.5, math.inf):
        grads = _grads(sizes, len(sizes))
        limit = _norm(grads) * factor if factor < math.inf else math.inf
        out = [torch.empty_like(g) for g in grads]
        _check_clip(specv, grads, limit, out=out)
        _check_clip(specv, grads, limit)


def test_clip_views_offsets_and_shapes(specv):
    flat32, flat16 = _randn((200000,), 3, 1.0), _randn((200000,), 4, 1.0).to(torch.bfloat16)
    grads = [flat32[1:1000], flat32[1003:90002], flat16[3:4], flat16[5:50001].view(2, -1),
             flat16[50001:50003], flat32[100001:100009].view(2, 2, 2), flat16[60000:199999]]
    keep = (flat32.clone(), flat16.clone())
    out32, out16 = torch.zeros_like(flat32), torch.zeros_like(flat16)
    out = [out32[3:1002], grads[1], out16[0:1], out16[1:49997].view(2, -1), out16[50001:50003],
           out32[100000:100008].view(2, 2, 2), out16[60001:200000]]
    before = [g.clone() for g in grads]
    want = _norm(before)
    specv.clip_grads(grads, want / 2, out=out)
    torch.cuda.synchronize()
    for b, o in zip(before, out):
        ref.close(o, b.double() * 0.5, (CLIP_EPS + 1e-6 + ref.out_u(b.dtype)) * b.double().abs(), "out")
    # what lies between and beside the gradients is untouched
    assert torch.equal(flat16, keep[1])
    assert torch.equal(flat32[1000:1003], keep[0][1000:1003])
    assert torch.equal(flat32[90002:], keep[0][90002:]) and flat32[0] == keep[0][0]
    used = torch.zeros(200000, dtype=torch.bool, device=DEV)
    for a, n in ((0, 1), (1, 49996), (50001, 2), (60001, 139999)):
        used[a:a + n] = True
    assert bool((out16[~used] == 0).all())


def test_clip_edges(specv):
    assert float(specv.clip_grads([], 1.0)) == 0.0
    assert float(specv.clip_grads([torch.empty(0, device=DEV)], 1.0)) == 0.0
    z = [torch.zeros(1000, device=DEV)]
    assert float(specv.clip_grads(z, 0.0)) == 0.0 and bool((z[0] == 0).all())
    g = _grads((3000, 70000), 5)
    specv.clip_grads(g, 0.0)
    assert all(bool((x == 0).all()) for x in g)
    # a norm that is not finite leaves the values as they are
    for bad in (float("nan"), math.inf, -math.inf, 3e38):
        g = _grads((3000, 70000), 6)
        g[0][17] = bad
        keep = [x.clone() for x in g]
        out = [torch.zeros_like(x) for x in g]
        n1 = float(specv.clip_grads(g, 1e-3, out=out))
        n2 = float(specv.clip_grads(g, 1e-3))
        assert not math.isfinite(n1) and not math.isfinite(n2)
        for x, k, o in zip(g, keep, out):
            same = lambda p, q: bool(((p == q) | (torch.isnan(p) & torch.isnan(q))).all())
            assert same(x, k) and same(o, k)


# --------------------------------------------------------- repeatability and streams
def test_scoring_is_repeatable(specv):
    zt, zq = _pair((6, 5, 50001), "bf16", 9)
    x = _tokens((6, 6), 50001, 1, 0.2)
    w = _weights((6, 5), 2, 0.2)
    g = _grads((1 << 20, 33, 700001), 3)
    runs = []
    for _ in range(3):
        lp = specv.token_logprobs(zt, x, top_n=8)
        loss, grad = specv.distill(zt, zq, w)
        out = [torch.empty_like(t) for t in g]
        norm = specv.clip_grads(g, 0.5, out=out)
        runs.append([*lp, loss, grad, norm, *out])
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_scoring_on_another_stream_and_in_a_graph(specv):
    zt, zq = _pair((2, 4, 30001), "bf16", 9)
    x = _tokens((2, 5), 30001, 1, 0.2)
    g = _grads((100000, 33), 3)
    out = [torch.empty_like(t) for t in g]

    def call(stream=None):
        lp = specv.token_logprobs(zt, x, top_n=8, stream=stream)
        gl = specv.token_logprobs_backward(zt, x, lp.stats, lp.entropy, lp.logprobs, None,
                                           stream=stream)
        loss, grad = specv.distill(zt, zq, stream=stream)
        norm = specv.clip_grads(g, 0.5, out=out, stream=stream)
        return [*lp, gl, loss, grad, norm]

    want = [t.clone() for t in call() + out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got + out))
    graph = torch.cuda.CUDAGraph()
    fresh = torch.cuda.Stream()  # a stream without a workspace yet
    fresh.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=fresh):
        got = call()
    for t in got + out:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got + out))


def test_scoring_offsets_past_32_bits(specv):
    """Element offsets past 2^31 in a strided view, and a gradient of more than
    2^31 entries."""
    V, sb = 5001, (1 << 30) + 5
    buf = torch.empty(2 * sb + 2 * V, dtype=torch.bfloat16, device=DEV)
    z = buf.as_strided((3, 2, V), (sb, V, 1))
    z.copy_(_randn((3, 2, V), 3))
    x = _tokens((3, 2), V, 4)
    got = _check_logprobs(specv, z, x, 5)
    g = _randn((3, 2), 5, 1.0)
    grad = specv.token_logprobs_backward(z, x, got.stats, got.entropy, g)
    want, tol = ref.logprobs_gradient(z, x, g, torch.zeros_like(g))
    ref.close(grad, want, tol, "gradient")
    _check_distill(specv, z, z[:, :2] * 0.5, None, 0)
    del buf, z
    B, V = 16500, 131072
    zq = torch.empty((B, 1, V), dtype=torch.bfloat16, device=DEV)
    for b in range(0, B, 500):
        zq[b:b + 500] = _randn((500, 1, V), b, 2.0).to(torch.bfloat16)
    zt = _randn((1, 1, V), 7, 2.0).to(torch.bfloat16).expand(B, 1, V)
    loss, grad = specv.distill(zt, zq)
    for b in (0, 8191, B - 1):
        rl, rg, lt, gt = ref.distill(zt[b:b + 1], zq[b:b + 1], torch.ones((1, 1), device=DEV), False)
        ref.close(loss[b:b + 1], rl, lt, "loss")
        ref.close(grad[b:b + 1], rg, gt, "gradient")
    x = torch.zeros((B, 1), dtype=torch.int32, device=DEV)
    fwd = specv.token_logprobs(zq, x, top_n=2)
    gl = specv.token_logprobs_backward(zq, x, fwd.stats, fwd.entropy, torch.ones((B, 1), device=DEV),
                                       out=grad)
    for b in (0, 8191, B - 1):
        want, tol = ref.logprobs_gradient(zq[b:b + 1], x[b:b + 1], torch.ones((1, 1), device=DEV),
                                          torch.zeros((1, 1), device=DEV))
        ref.close(gl[b:b + 1], want, tol, "gradient")


def test_scoring_many_short_rows(specv):
    """More rows than a grid has CTAs at once."""
    R, V = 70001, 33
    z = _randn((R, V), 3)
    x = _tokens((R,), V, 4, 0.1)
    got = specv.token_logprobs(z, x, top_n=2)
    lp = torch.log_softmax(z.double(), -1)
    live = x >= 0
    want = lp.gather(-1, x.clamp_min(0).long().unsqueeze(-1)).squeeze(-1).where(live, torch.zeros(()).double().to(DEV))
    ref.close(got.logprobs, want, 64 * ref.U * (8 + want.abs()), "logprobs")
    best = z.argmax(-1).where(live, torch.full_like(x, -1).long())
    assert torch.equal(got.top_tokens[:, 0].long(), best)
    zt = _randn((R, 1, V), 5)
    loss, grad = specv.distill(zt, z.unsqueeze(1))
    rl, rg, lt, gt = ref.distill(zt, z.unsqueeze(1), torch.ones((R, 1), device=DEV), False)
    ref.close(loss, rl, lt, "loss")
    ref.close(grad, rg, gt, "gradient")


# ---------------------------------------------------------------------- refusals
def test_scoring_refuses_bad_tensors(specv):
    z, x = _randn((2, 3, 50), 1), _tokens((2, 3), 50, 1)
    f = torch.zeros((2, 3), device=DEV)
    for bad in (dict(logits=z.half()), dict(tokens=x.long()), dict(logits=z.cpu(), tokens=x.cpu())):
        with pytest.raises((TypeError, ValueError)):
            specv.token_logprobs(bad.get("logits", z), bad.get("tokens", x))
    for call in (lambda: specv.token_logprobs(z, x, top_n=33),
                 lambda: specv.token_logprobs(z, x, top_n=-1),
                 lambda: specv.token_logprobs(z, x[:, :2]),
                 lambda: specv.token_logprobs(z.transpose(1, 2), x),
                 lambda: specv.token_logprobs(z[0, 0], x[0, 0]),
                 lambda: specv.token_logprobs_backward(z, x, f, f, f),
                 lambda: specv.token_logprobs_backward(z, x, torch.zeros((2, 3, 2), device=DEV), f,
                                                       f, out=torch.empty_like(z)[:, :, ::1][:1]),
                 lambda: specv.distill(z, z[:, :1]), lambda: specv.distill(z[:1], z),
                 lambda: specv.distill(z, z, weight=f[:1]), lambda: specv.distill(z, z, kind=2),
                 lambda: specv.distill(z, z, out_grad=torch.empty((2, 3, 60), device=DEV)[..., :50]),
                 lambda: specv.clip_grads([z], -1.0), lambda: specv.clip_grads([z], float("nan")),
                 lambda: specv.clip_grads([z.transpose(0, 1)], 1.0),
                 lambda: specv.clip_grads([z, z], 1.0), lambda: specv.clip_grads([z.cpu()], 1.0),
                 lambda: specv.clip_grads([z], 1.0, out=[]),
                 lambda: specv.clip_grads([z], 1.0, out=[torch.empty(7, device=DEV)])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        specv.distill(z.bfloat16(), z)
    with pytest.raises(TypeError):
        specv.clip_grads([z.half()], 1.0)
    odd = torch.zeros(13, device=DEV)[1:].view(2, 3, 2)  # contiguous, 4 bytes off a pair
    with pytest.raises(specv.SpecvError):
        specv.token_logprobs_backward(z, x, odd, f, f)
    with pytest.raises(specv.SpecvError):  # no rows
        specv.token_logprobs(z[:0], x[:0])
