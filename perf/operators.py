"""The operators that stand next to the verify step, as cases to be measured.

Three of them, on the data that a step of speculative decoding leaves behind:

* ``token_logprobs``: the log probability of each emitted token, with the entropy
  of its row and the most likely alternatives; and its gradient.
* ``distill``: the divergence of the draft's rows from the target's, with its
  gradient with respect to the draft logits.
* ``clip_grads``: the 2-norm over all gradients of the draft's weights, and
  clipping to a largest norm.

``run`` computes each in plain torch operations, or, where ``own`` is true, by
the library's calls; ``exact`` computes it in 64 bits from its definition.
"""
import math

import torch

own = False

DEV = "cuda"
NEG = -math.inf


# --------------------------------------------------------------------- cases
def _logprobs(name, B, N, V, dtype, top, skip=0.0, pad=0, masked=0):
    return dict(name=name, op="logprobs", B=B, N=N, V=V, dtype=dtype, top=top, skip=skip, pad=pad,
                masked=masked)


def _backward(name, B, N, V, dtype, skip=0.0, pad=0, masked=0):
    return dict(name=name, op="backward", B=B, N=N, V=V, dtype=dtype, skip=skip, pad=pad,
                masked=masked)


def _distill(name, B, N, V, dtype, kind, skip=0.0, pad=0, masked=0):
    return dict(name=name, op="distill", B=B, N=N, V=V, dtype=dtype, kind=kind, skip=skip, pad=pad,
                masked=masked)


def _clip(name, tensors, largest, f32_share, clipped):
    return dict(name=name, op="clip", tensors=tensors, largest=largest, f32_share=f32_share,
                clipped=clipped)


def listed():
    return [
        # one request's step: nine positions of one sequence; the call's latency counts
        _logprobs("logprobs one step", 1, 9, 128256, "bf16", 5),
        # a served batch: the positions after each first rejection hold no token; as many
        # alternatives as serving interfaces offer
        _logprobs("logprobs served batch", 32, 6, 152064, "bf16", 20, skip=0.5, masked=64),
        # a large batch scored whole, as for an evaluation or for training data
        _logprobs("logprobs large batch", 256, 9, 128256, "f32", 1),
        # a vocabulary that no vector divides, rows off every boundary
        _logprobs("logprobs odd vocabulary", 37, 5, 100003, "bf16", 5, masked=3),
        # a small vocabulary (bytes, characters) in training
        _backward("gradient small vocabulary", 512, 8, 1000, "f32", skip=0.1),
        # a training batch over a large vocabulary
        _backward("gradient large batch", 256, 8, 128256, "bf16", skip=0.1),
        # a few short rows: the call's latency counts
        _distill("distill short rows", 8, 4, 1000, "f32", "forward"),
        # what a served batch leaves for the draft's fitting
        _distill("distill served batch", 32, 5, 152064, "bf16", "forward", skip=0.25, masked=64),
        # a training batch, 32-bit logits
        _distill("distill large batch", 256, 8, 128256, "f32", "forward"),
        # the other divergence; odd vocabulary, masked padding, left-out positions
        _distill("distill odd vocabulary", 19, 7, 50001, "bf16", "reverse", skip=0.2, masked=17),
        # a draft head's few gradients, below the limit: the common step, nothing to scale
        _clip("clip draft head", 14, 2_000_000, 0.3, False),
        # a whole draft model's gradients, over the limit
        _clip("clip draft model", 290, 16_000_000, 0.25, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST_BYTES = 1.0e9


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "backward", "distill", "distill", "clip"])
    if op == "clip":
        tensors = _log(rng, 3, 300)
        largest = _log(rng, 20_000, 16_000_000)
        return _drawn(_clip("", tensors, largest, round(rng.random(), 2), rng.random() < 0.6))
    dtype = rng.choice(["f32", "bf16"])
    V = _log(rng, 500, 152064)
    # a round width, an odd one, or an even one off the round widths
    V = rng.choice([V // 128 * 128 + 64, V | 1, V // 128 * 128 + 2 * rng.randint(1, 63)])
    N = rng.randint(1, 16)
    e = 4 if dtype == "f32" else 2
    B = _log(rng, 1, max(2, min(4096, int(_MOST_BYTES / (3.0 * e * V * (N + 1))))))
    skip = rng.choice([0.0, 0.25, 0.5])
    pad = rng.choice([0, 0, rng.randint(1, 128)])
    masked = rng.choice([0, rng.randint(1, 100)])
    if op == "logprobs":
        return _drawn(_logprobs("", B, N, V, dtype, rng.choice([0, 1, 3, 5, 10, 20, 32]), skip, pad,
                                masked))
    if op == "backward":
        return _drawn(_backward("", B, N, V, dtype, skip, pad, masked))
    return _drawn(_distill("", B, N, V, dtype, rng.choice(["forward", "reverse"]), skip, pad, masked))


def _drawn(case):
    case.pop("name")
    return case


# -------------------------------------------------------------------- inputs
def _gen(seed, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + k)
    return g


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _rows(B, N, V, dtype, pad, masked, values):
    """Rows of V logits in a buffer whose rows are V + pad apart (an output layer padded
    to a round width); the last `masked` entries of the vocabulary are padding: -inf."""
    buf = torch.zeros((B, N, V + pad), dtype=dtype, device=DEV)
    z = buf[..., :V]
    z.copy_(values)
    if masked:
        z[..., V - masked:] = NEG
    return z


def _sizes(case):
    """The tensors of a draft's gradients: matrices and vectors, of many sizes, some odd."""
    n, largest = case["tensors"], case["largest"]
    out = []
    for i in range(n):
        kind = i % 7
        if kind in (0, 3):
            size = largest // (1 + i % 4)
        elif kind in (1, 4):
            size = largest // 8 + 3 * i
        elif kind == 2:
            size = max(1, largest // 4096)
        elif kind == 5:
            size = 1 + i * 37 % 1000
        else:
            size = largest // 64 + 1
        out.append((max(1, size), (i * 61 % 100) < 100 * case["f32_share"]))
    return out


def _bytes_of(case):
    return sum(size * (4 if f32 else 2) for size, f32 in _sizes(case))


def prepare(case, seed):
    op = case["op"]
    if op == "clip":
        # gradients as views of two flat buffers, one for each type, each tensor's start on
        # a 16-byte boundary, as frameworks that bucket their gradients keep them
        sizes = _sizes(case)
        flat, at = {}, {True: 0, False: 0}
        places = []
        for size, f32 in sizes:
            places.append((f32, at[f32], size))
            at[f32] += -(-size // 8) * 8
        g = _gen(seed, 0)
        for f32 in (True, False):
            flat[f32] = torch.randn(max(8, at[f32]), generator=g, device=DEV,
                                    dtype=torch.float32 if f32 else torch.bfloat16).mul_(1e-2)
        used = {f32: torch.zeros(flat[f32].numel(), dtype=torch.bool, device=DEV) for f32 in flat}
        for f32, a, size in places:
            used[f32][a:a + size] = True
        for f32 in flat:
            flat[f32].masked_fill_(~used[f32], 0)
        del used
        norm = 1e-2 * math.sqrt(sum(size for size, _ in sizes))  # about
        out = {k: torch.zeros_like(v) for k, v in flat.items()} if case["clipped"] else flat
        return dict(case=case, grads=[flat[f][a:a + s] for f, a, s in places],
                    out=[out[f][a:a + s] for f, a, s in places], flat=[out[True], out[False]],
                    max_norm=norm * (0.5 if case["clipped"] else 2.0))
    B, N, V, dtype = case["B"], case["N"], case["V"], _dtype(case)
    s = dict(case=case)
    if op == "distill":
        zt = torch.randn((B, N + 1, V), generator=_gen(seed, 0), device=DEV).mul_(3.0)
        s["target"] = _rows(B, N + 1, V, dtype, 0, case["masked"], zt)
        zq = torch.randn((B, N, V), generator=_gen(seed, 1), device=DEV)
        zq.add_(zt[:, :N], alpha=0.85)
        s["draft"] = _rows(B, N, V, dtype, case["pad"], case["masked"], zq)
        w = torch.rand((B, N), generator=_gen(seed, 2), device=DEV) + 0.5
        live = torch.rand((B, N), generator=_gen(seed, 3), device=DEV) >= case["skip"]
        s["weight"] = w * live
        return s
    z = torch.randn((B, N, V), generator=_gen(seed, 0), device=DEV).mul_(3.0)
    s["logits"] = _rows(B, N, V, dtype, case["pad"], case["masked"], z)
    del z
    # most emitted tokens are likely ones; some come from far down
    k = max(1, V - case["masked"])
    best = s["logits"].float().argmax(-1)
    far = torch.randint(0, k, (B, N), generator=_gen(seed, 1), device=DEV)
    pick = torch.rand((B, N), generator=_gen(seed, 2), device=DEV)
    tokens = torch.where(pick < 0.5, best, far)
    live = torch.rand((B, N), generator=_gen(seed, 3), device=DEV) >= case["skip"]
    s["tokens"] = torch.where(live, tokens, torch.full_like(tokens, -1)).to(torch.int32)
    if op == "backward":
        s["stats"], s["entropy"] = _row_stats(s["logits"], s["tokens"])
        s["g"] = torch.randn((B, N), generator=_gen(seed, 4), device=DEV)
        s["h"] = torch.randn((B, N), generator=_gen(seed, 5), device=DEV).mul_(0.1)
    return s


def _row_stats(logits, tokens):
    """What the forward call leaves for its gradient: (max, ln sum exp(z - max)) and the entropy."""
    B, N, V = logits.shape
    stats = torch.empty((B, N, 2), dtype=torch.float32, device=DEV)
    entropy = torch.empty((B, N), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (N * V))
    for b in range(0, B, step):
        z = logits[b:b + step].double()
        m = z.amax(-1, keepdim=True)
        d = z - m
        e = d.exp()
        total = e.sum(-1)
        stats[b:b + step, :, 0] = m[..., 0].float()
        stats[b:b + step, :, 1] = total.log().float()
        entropy[b:b + step] = (total.log() - (e * d.clamp_min(-1e4)).sum(-1) / total).float()
    dead = tokens < 0
    stats[dead] = 0
    entropy[dead] = 0
    return stats, entropy


# ----------------------------------------------------------------- plain form
def _plain_logprobs(logits, tokens, top):
    V = logits.shape[-1]
    live = tokens >= 0
    z = logits.float()
    m = z.amax(-1)
    d = z - m.unsqueeze(-1)
    e = d.exp()
    total = e.sum(-1)
    ln = total.log()
    entropy = ln - (e * d.clamp_min(-1e4)).sum(-1) / total
    zx = z.gather(-1, tokens.clamp_min(0).long().unsqueeze(-1)).squeeze(-1)
    zero = torch.zeros_like(m)
    out = dict(logprobs=torch.where(live, (zx - m) - ln, zero),
               entropy=torch.where(live, entropy, zero),
               stats=torch.stack([torch.where(live, m, zero), torch.where(live, ln, zero)], -1))
    if top:
        # one whole number for each entry, larger for the larger value, then for the lower index
        bits = (z + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = order * 2**32 + (2**32 - 1 - torch.arange(V, device=z.device))
        at = 2**32 - 1 - (key.topk(top, dim=-1).values & 0xFFFFFFFF)
        value = z.gather(-1, at)
        fine = live.unsqueeze(-1) & (value > NEG)
        out["top_tokens"] = torch.where(fine, at, torch.full_like(at, -1)).to(torch.int32)
        out["top_logprobs"] = torch.where(fine, (value - m.unsqueeze(-1)) - ln.unsqueeze(-1),
                                          torch.full_like(value, NEG))
    return out


def _plain_backward(logits, tokens, stats, entropy, g, h):
    live = (tokens >= 0).unsqueeze(-1)
    lnp = (logits.float() - stats[..., :1]) - stats[..., 1:]
    p = lnp.exp()
    grad = -p * (g.unsqueeze(-1) + h.unsqueeze(-1) * (lnp.clamp_min(-1e4) + entropy.unsqueeze(-1)))
    at = tokens.clamp_min(0).long().unsqueeze(-1)
    grad.scatter_add_(-1, at, g.unsqueeze(-1))
    return torch.where(live, grad, torch.zeros_like(grad)).to(logits.dtype)


def _plain_distill(target, draft, weight, kind):
    K = draft.shape[1]
    zt, zq = target[:, :K].float(), draft.float()
    lp = zt - zt.amax(-1, keepdim=True)
    lp = lp - lp.exp().sum(-1, keepdim=True).log()
    lq = zq - zq.amax(-1, keepdim=True)
    lq = lq - lq.exp().sum(-1, keepdim=True).log()
    p, q = lp.exp(), lq.exp()
    w = weight.unsqueeze(-1)
    if kind == "forward":
        loss = torch.where(p > 0, p * (lp - lq), torch.zeros_like(p)).sum(-1)
        grad = w * (q - p)
    else:
        r = torch.where(q > 0, lq - lp, torch.zeros_like(q))
        loss = (q * r).sum(-1)
        grad = w * (q * (r - loss.unsqueeze(-1)))
    return dict(loss=weight * loss, grad=grad.to(draft.dtype))


def _plain_clip(grads, out, max_norm):
    norm = torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()
    c = (max_norm / (norm + 1e-6)).clamp_max(1.0)
    _ = [o.copy_(g.float() * c) for g, o in zip(grads, out)]
    return norm


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import speculative_decoding_verification_specv_gb300 as specv
        if op == "logprobs":
            return specv.token_logprobs(state["logits"], state["tokens"],
                                        top_n=case["top"])._asdict()
        if op == "backward":
            return specv.token_logprobs_backward(state["logits"], state["tokens"], state["stats"],
                                                 state["entropy"], state["g"], state["h"])
        if op == "distill":
            kind = specv.FORWARD_KL if case["kind"] == "forward" else specv.REVERSE_KL
            loss, grad = specv.distill(state["target"], state["draft"], state["weight"], kind=kind)
            return dict(loss=loss, grad=grad)
        norm = specv.clip_grads(state["grads"], state["max_norm"], out=state["out"])
        return dict(norm=norm, grads=state["flat"])
    if op == "logprobs":
        return _plain_logprobs(state["logits"], state["tokens"], case["top"])
    if op == "backward":
        return _plain_backward(state["logits"], state["tokens"], state["stats"], state["entropy"],
                               state["g"], state["h"])
    if op == "distill":
        return _plain_distill(state["target"], state["draft"], state["weight"], case["kind"])
    norm = _plain_clip(state["grads"], state["out"], state["max_norm"])
    return dict(norm=norm, grads=state["flat"])


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = 0.0
        for g in s["grads"]:
            x = g.double()
            total += float((x * x).sum())
        norm = math.sqrt(total)
        c = min(1.0, s["max_norm"] / (norm + 1e-6))
        flat = [torch.zeros(f.numel(), dtype=torch.float64, device=DEV) for f in s["flat"]]
        for g, o in zip(s["grads"], s["out"]):
            to = flat[0] if g.dtype == torch.float32 else flat[1]
            at = o.storage_offset()
            to[at:at + g.numel()] = g.double() * c
        return dict(norm=norm, grads=flat)
    if op == "distill":
        B, K, V = s["draft"].shape
        loss = torch.empty((B, K), dtype=torch.float64, device=DEV)
        grad = torch.empty((B, K, V), dtype=torch.float64, device=DEV)
        for b in range(B):
            t, q = s["target"][b, :K].double(), s["draft"][b].double()
            w = s["weight"][b].double()
            lt = t - torch.logsumexp(t, -1, keepdim=True)
            lq = q - torch.logsumexp(q, -1, keepdim=True)
            a, c = (lt, lq) if case["kind"] == "forward" else (lq, lt)
            term = a.exp() * (a - c)
            term[a == NEG] = 0.0
            kl = term.sum(-1)
            if case["kind"] == "forward":
                d = lq.exp() - lt.exp()
            else:
                d = term - lq.exp() * kl.unsqueeze(-1)
            loss[b] = w * kl
            grad[b] = w.unsqueeze(-1) * d
        return dict(loss=loss, grad=grad)
    B, N, V = s["logits"].shape
    if op == "backward":
        grad = torch.zeros((B, N, V), dtype=torch.float64, device=DEV)
        for b in range(B):
            z = s["logits"][b].double()
            lp = z - torch.logsumexp(z, -1, keepdim=True)
            p = lp.exp()
            plp = p * lp
            plp[p == 0] = 0.0
            H = -plp.sum(-1, keepdim=True)
            g, h = s["g"][b].double().unsqueeze(-1), s["h"][b].double().unsqueeze(-1)
            d = -g * p - h * (plp + p * H)
            x = s["tokens"][b].long()
            d[torch.arange(N, device=DEV), x.clamp_min(0)] += g[:, 0]
            d[x < 0] = 0.0
            grad[b] = d
        return grad
    top = case["top"]
    out = dict(logprobs=torch.zeros((B, N), dtype=torch.float64, device=DEV),
               entropy=torch.zeros((B, N), dtype=torch.float64, device=DEV),
               stats=torch.zeros((B, N, 2), dtype=torch.float64, device=DEV))
    if top:
        out["top_tokens"] = None
        out["top_logprobs"] = torch.full((B, N, top), NEG, dtype=torch.float64, device=DEV)
    for b in range(B):
        x = s["tokens"][b].long()
        live = x >= 0
        z = s["logits"][b].double()
        lse = torch.logsumexp(z, -1)
        lp = z - lse.unsqueeze(-1)
        plp = lp.exp() * lp
        plp[lp == NEG] = 0.0
        m = z.max(-1).values
        out["logprobs"][b] = torch.where(live, lp[torch.arange(N, device=DEV), x.clamp_min(0)], 0.0)
        out["entropy"][b] = torch.where(live, -plp.sum(-1), 0.0)
        out["stats"][b, :, 0] = torch.where(live, m, 0.0)
        out["stats"][b, :, 1] = torch.where(live, lse - m, 0.0)
        if top:
            best = lp.sort(-1, descending=True).values[:, :top]
            out["top_logprobs"][b] = torch.where(live.unsqueeze(-1), best, NEG)
    return out


# ------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "clip":
        n = sum(size for size, _ in _sizes(case))
        reads = _bytes_of(case)
        return dict(bytes=reads * (2 if case["clipped"] else 1), flops=(3 if case["clipped"] else 2) * n)
    e = 4 if case["dtype"] == "f32" else 2
    R, V = case["B"] * case["N"], case["V"]
    live = R * (1.0 - case["skip"])
    if case["op"] == "logprobs":
        return dict(bytes=live * V * e + R * (4 + 16 + 8 * case["top"]), flops=6 * live * V)
    if case["op"] == "backward":
        return dict(bytes=(live + R) * V * e + R * 24, flops=8 * live * V)
    return dict(bytes=(2 * live + R) * V * e + R * 8, flops=16 * live * V)
