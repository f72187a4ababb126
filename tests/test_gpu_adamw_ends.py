"""GPU tests of adamw_step at the ends of its ranges: blocks of 8-bit roots that lie far
apart, graphs that saved a weight, norms near fp32's largest,
squares below its normal numbers."""
import math

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


@pytest.mark.parametrize("n", [1024, 1021])
@pytest.mark.parametrize("large", [1e3, 5e5, 1e6, 1e9, 1e15])
def test_small_roots_beside_large_ones(specv, large, n):
    """A root that is not 0 is stored as the smallest positive value at least: its weight would
    move by m / eps otherwise.  From zero states the root is sqrt(1 - beta2) |g|; gradients from
    2^-57 on have squares, times 1 - beta2, of at least 2^-124, in fp32's normal numbers, so
    their roots are not 0.  The second block has no large one; the third only zeros."""
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, device=DEV)
    sizes = 2.0 ** -torch.arange(0, 57.5, 0.5, device=DEV)
    g[:256:2] = sizes.repeat(3)[:128]
    g[100], g[32] = large, -large
    g[256:512:2] = sizes.repeat(3)[:128]
    g[700:] = 0
    st = specv.adamw_state([p], 8)
    for t in (1, 2, 3):
        specv.adamw_step([p], [g], st, t, 1e-3, seed=t)
        torch.cuda.synchronize()
        codes = st.exp_avg_sq[0].view(torch.uint8)
        assert bool((codes[g != 0] >= 1).all()), int((codes[g != 0] == 0).sum())
        assert bool((codes[g == 0] == 0).all())
        # smaller than the smallest value by far: exactly that one
        far = (g != 0) & (torch.arange(n, device=DEV) < 256) & (g.abs() < large * 2.0 ** -30)
        assert bool((codes[far] == 1).all()) and (int(far.sum()) > 0 or large < 1e4)
        s = st.scales[0][:, 1].double()
        want = large * math.sqrt(1 - 0.999 ** t) / 448
        assert abs(float(s[0]) - want) <= want * 2.0 ** -4  # (the stored root is rounded each step)


def test_a_graph_that_saved_a_weight_refuses_to_go_back(specv):
    """As with any step in place: its gradients would be those of other weights."""
    x = torch.ones((4, 3), device=DEV, requires_grad=True)
    w = torch.nn.Parameter(torch.ones((5, 3), device=DEV))
    y = (x @ w.T).square().sum()
    y.backward(retain_graph=True)
    st = specv.adamw_state([w])
    specv.adamw_step([w], [w.grad], st, 1, 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    z = torch.randn((2, 50), device=DEV, requires_grad=True)
    rows = z * 1.0
    loss = rows.square().sum()
    specv.filter_logits(rows.detach(), top_k=3, out=rows.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # a step after the backward pass is what a training loop does
    for t in (2, 3):
        w.grad = None
        (x @ w.T).square().sum().backward()
        specv.adamw_step([w], [w.grad], st, t, 0.1)


@pytest.mark.parametrize("max_norm", [math.inf, 1e39, torch.finfo(torch.float32).max])
def test_a_limit_that_no_norm_exceeds(specv, max_norm):
    """min(1, max_norm / (norm + 1e-6)) is 1 for any finite norm."""
    n = 3000
    for norm in (torch.finfo(torch.float32).max, 3.39e38, 1.0, 0.0):
        both = []
        for kw in (dict(), dict(norm=torch.tensor(norm, device=DEV), max_norm=max_norm)):
            p = [torch.linspace(-1, 1, n, device=DEV)]
            g = [torch.linspace(-3e-3, 2e-3, n, device=DEV)]
            st = specv.adamw_state(p)
            specv.adamw_step(p, g, st, 1, 0.1, **kw)
            both.append((p[0], st.exp_avg[0], st.exp_avg_sq[0]))
        for x, y in zip(*both):
            assert torch.equal(x, y), norm


def test_under_inference_mode(specv):
    """Tensors made there have no version counters to move."""
    with torch.inference_mode():
        p, g = [torch.ones(3000, device=DEV)], [torch.full((3000,), 0.5, device=DEV)]
        st = specv.adamw_state(p)
        specv.adamw_step(p, g, st, 1, 0.1)
        z, u = torch.randn((4, 5000), device=DEV), torch.rand(4, device=DEV)
        want = specv.filter_logits(z, top_k=9)
        drawn = specv.sample_tokens(z, u, top_k=9, out_filtered=z)
        again = specv.filter_logits(z, top_k=9, out=z)
    w = torch.ones(3000, device=DEV)  # (an ordinary tensor too)
    with torch.inference_mode():
        specv.adamw_step([w], g, specv.adamw_state([w]), 1, 0.1)
    torch.cuda.synchronize()
    assert bool(((p[0] - 0.9).abs() <= 1e-6).all()) and torch.equal(w, p[0])
    assert torch.equal(z, want) and again is z
    assert bool((want.gather(-1, drawn.tokens.long().unsqueeze(-1)) > -math.inf).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_squares_below_the_normal_numbers(specv, bits):
    """With eps = 0 the first step is the rate against the gradient's sign whatever its size.  v
    is off by half of fp32's smallest spacing, 2^-150, besides its roundings, its root by half
    of that in proportion: the weight (0 before) by that much of the rate and some 2^-20."""
    for k in range(40, 67):
        g = torch.full((600,), 2.0 ** -k, device=DEV)
        g[::3] *= -1.0
        p = torch.zeros(600, device=DEV)
        st = specv.adamw_state([p], bits)
        specv.adamw_step([p], [g], st, 1, 0.25, eps=0.0)
        v = 1e-3 * 2.0 ** (-2 * k)
        tol = 0.25 * (0.5 * 2.0 ** -150 / v * (1 + 2.0 ** -7) + 2.0 ** -20)
        assert float((p + 0.25 * g.sign()).abs().max()) <= tol, k
        if bits == 8:
            assert bool((st.exp_avg_sq[0].float() == 448).all())
