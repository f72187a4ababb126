"""GPU test of sample_tokens and filter_logits on rows that another stream writes meanwhile:
what comes out of such a call is not defined, but tokens lie within the row, nothing around
the outputs is written, and the next call is right."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("R,V", [(300, 1000), (700, 5003), (320, 20011), (152, 128256)], ids=str)
def test_rows_written_meanwhile(specv, R, V, dtype):
    g = torch.Generator(device=DEV).manual_seed(V)
    base = (torch.randn((R, V), generator=g, device=DEV) * 2).to(dtype)
    others = [base * 0.01, base.flip(-1) * 40 + 1000, -base.abs() * 1e30, base + math.inf,
              torch.full_like(base, float("nan")), torch.full_like(base, -math.inf)]
    z = base.clone()
    u = torch.rand((R,), generator=g, device=DEV)
    guarded = torch.full((R * V + 64,), 3.0, dtype=dtype, device=DEV)
    out = guarded[32:32 + R * V].view(R, V)
    filters = [dict(), dict(top_k=40), dict(top_p=0.95), dict(top_k=V // 3, top_p=0.9),
               dict(top_k=V // 2), dict(min_p=0.05), dict(top_p=0.5, min_p=1e-4)]
    want = [(specv.sample_tokens(z, u, 0.8, **kw), specv.filter_logits(z, 0.8, **kw)) for kw in filters]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    found = []
    for kw in filters:
        with torch.cuda.stream(side):
            for _ in range(6):
                for x in others:
                    z.copy_(x)
        for _ in range(8):
            found.append(specv.sample_tokens(z, u, 0.8, out_filtered=out, **kw).tokens)
    torch.cuda.synchronize()
    for x in found:
        assert bool(((x >= -1) & (x < V)).all())
    assert bool((guarded[:32] == 3).all()) and bool((guarded[32 + R * V:] == 3).all())
    z.copy_(base)
    for kw, (a, f) in zip(filters, want):
        b = specv.sample_tokens(z, u, 0.8, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b)), kw
        assert torch.equal(specv.filter_logits(z, 0.8, **kw), f), kw
