"""64-bit restatements of the operators on the step's logits, and the error that
32-bit kernels may make, derived below from the operations they perform.

Bounds (u = 2^-24, half an ulp of fp32).  A row sum of V positive terms: a thread
adds at most L = ceil(V / 32) terms one after the other (32 threads at least serve
a row), the partials are merged in at most 64 further additions and rescalings, and
each term e^d carries the error of the fp32 exponential (2 ulp, and u |d log2 e|
from rounding its argument; weighted by e^d, |d| e^d <= 1, at most a few u).  So a
sum's relative error is at most eps_S = (L + 64) u.  Everything below is a multiple
of it plus the roundings of the last few operations.
"""
import math

import torch

U = 2.0 ** -24
NEG = float("-inf")


def eps_sum(V):
    return (-(-V // 32) + 64) * U


def out_u(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2 * U


def token_logprobs(logits, tokens, top_n):
    """(logprob, entropy, max, ln sum, top tokens, top logprobs, tolerance) in
    64 bits, on the CPU, for logits [..., V] of any type."""
    z = logits.detach().cpu().double()
    lead, V = z.shape[:-1], z.shape[-1]
    z = z.reshape(-1, V)
    x = tokens.detach().cpu().long().reshape(-1)
    R = z.shape[0]
    f64 = dict(dtype=torch.float64)
    lp_x, H = torch.zeros(R, **f64), torch.zeros(R, **f64)
    M, ln = torch.zeros(R, **f64), torch.zeros(R, **f64)
    tt = torch.full((R, top_n), -1, dtype=torch.int32)
    tl = torch.full((R, top_n), NEG, **f64)
    tol = torch.zeros(R, **f64)
    nan = float("nan")
    for r in range(R):
        t = int(x[r])
        if t == -1:
            continue
        row = z[r]
        if t < 0 or t >= V or bool(torch.isnan(row).any()) or bool((row == math.inf).any()):
            lp_x[r] = H[r] = M[r] = ln[r] = nan
            tl[r] = nan
            continue
        m = row.max()
        M[r] = m
        if m == NEG:
            lp_x[r] = NEG
            continue
        d = row - m
        e = d.exp()
        s = e.sum()
        ln[r] = s.log()
        mean = float((e * d.clamp_min(-1e6)).sum() / s)
        lp_x[r] = d[t] - ln[r]
        H[r] = ln[r] - mean
        value, at = row.sort(descending=True, stable=True)
        k = min(top_n, V)
        fine = value[:k] > NEG
        tt[r, :k] = torch.where(fine, at[:k], -1).to(torch.int32)
        tl[r, :k] = torch.where(fine, value[:k] - m - ln[r], NEG)
        # ln S errs by eps_S; T / S by eps_S times the mean |d|, and recentring a
        # partial whose reference lies up to 16 below adds 16 eps_S
        tol[r] = eps_sum(V) * (18 - 2 * mean) + 4 * U * (1 + abs(mean) + float(ln[r]))
    shape = lambda t: t.reshape(*lead, *t.shape[1:])
    return tuple(shape(t) for t in (lp_x, H, M, ln, tt, tl, tol))


def logprobs_gradient(logits, tokens, g, h):
    """(gradient, tolerance of each entry) in 64 bits, on the logits' device."""
    z = logits.double()
    V = z.shape[-1]
    m = z.amax(-1, keepdim=True)
    d = z - m
    ln = d.exp().sum(-1, keepdim=True).log()
    lp = d - ln
    p = lp.exp()
    lp0 = lp.clamp_min(-1e6)
    H = -(p * lp0).sum(-1, keepdim=True)
    g, h = g.double().unsqueeze(-1), h.double().unsqueeze(-1)
    grad = -p * (g + h * (lp0 + H))
    at = tokens.clamp(0, V - 1).long().unsqueeze(-1)
    grad.scatter_add_(-1, at, g.expand_as(at).clone())
    # p errs by the roundings of its exponent, (|d| + ln S + 1) u times a few, by the
    # statistics' own error, and by the exponential's 2 ulp
    eps = U * (12 + 6 * lp0.abs() + 6 * ln) + eps_sum(V)
    size = p * (g.abs() + h.abs() * (lp0.abs() + H.abs() + 40))
    tol = eps * size + out_u(logits.dtype) * grad.abs() + 1e-36
    tol.scatter_add_(-1, at, (4 * U * g.abs()).expand_as(at).clone())
    dead = (tokens == -1) | (m.squeeze(-1) == NEG)
    bad = (tokens < -1) | (tokens >= V) | (~dead & ~torch.isfinite(ln.squeeze(-1)))
    grad[dead] = 0.0
    grad[bad] = float("nan")
    return grad, tol


def distill(target, draft, weight, reverse):
    """(loss, gradient, loss tolerance, gradient tolerance) in 64 bits for row pairs
    [..., V] and weights [...], on their device."""
    t, q = target.double(), draft.double()
    V = q.shape[-1]
    w = weight.double()
    dt, dq = t - t.amax(-1, keepdim=True), q - q.amax(-1, keepdim=True)
    st, sq = dt.exp().sum(-1, keepdim=True), dq.exp().sum(-1, keepdim=True)
    lt, lq = dt - st.log(), dq - sq.log()
    a, c = (lq, lt) if reverse else (lt, lq)
    # entries of positive leading probability; against a masked entry of the other row
    # only those that fp32 does not hold as zero (no test input lies near that limit)
    on = (a > NEG) & ((c > NEG) | ((dq if reverse else dt) > -80.0))
    diff = torch.where(on, a - c, torch.zeros_like(a))
    lead = torch.where(on, a.exp(), torch.zeros_like(a))
    kl = (lead * diff).sum(-1)
    wx = w.unsqueeze(-1)
    if reverse:
        grad = wx * (lq.exp() * torch.where(on, a - c - kl.unsqueeze(-1), torch.zeros_like(a)))
        inf = torch.isinf(kl).unsqueeze(-1) & on
        grad = torch.where(inf, torch.full_like(grad, float("nan")), grad)
    else:
        grad = wx * (lq.exp() - lt.exp())
    empty = (t.amax(-1) == NEG) | (q.amax(-1) == NEG) | (w == 0)
    bad = (torch.isnan(t) | (t == math.inf) | torch.isnan(q) | (q == math.inf)).any(-1) & (w != 0)
    loss = w * kl
    e = eps_sum(V)
    spread = (lead * diff.abs().clamp_max(1e6)).sum(-1)
    logs = st.log().squeeze(-1) + sq.log().squeeze(-1)
    kl_tol = e * (20 + 4 * spread) + 8 * U * (1 + spread + logs)
    loss_tol = w.abs() * kl_tol + 2 * U * loss.abs()
    far = lambda d, s: U * (12 + 6 * d.clamp_min(-1e6).abs() + 6 * s.log()) + e
    eq, et = lq.exp() * far(dq, sq), lt.exp() * far(dt, st)
    if reverse:
        size = diff.abs().clamp_max(1e6) + kl.abs().clamp_max(1e6).unsqueeze(-1)
        tol = wx.abs() * (eq * (size + 1) * 2 + lq.exp() * kl_tol.unsqueeze(-1))
    else:
        tol = wx.abs() * (eq + et)
    tol = tol + out_u(draft.dtype) * grad.abs().nan_to_num(0.0, 0.0, 0.0) + 1e-36
    loss = torch.where(empty, torch.zeros_like(loss), loss)
    grad[empty] = 0.0
    loss[bad] = float("nan")
    grad[bad] = float("nan")
    return loss, grad, loss_tol, tol


def close(got, ref, tol, what):
    """Every value within its tolerance; NaN and infinities in the same places."""
    got = got.double().to(ref.device)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    off = (got - ref).abs()
    ok = same | (torch.isfinite(ref) & (off <= tol))
    if not bool(ok.all()):
        i = (~ok).nonzero()[0].tolist()
        k = tuple(i)
        t = tol[k] if tol.dim() == ref.dim() else tol
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off; at {i} got "
                             f"{float(got[k])!r}, want {float(ref[k])!r} +- {float(t):.3g}")
