"""Fit a draft head to its target from the verify step's own logits.

    python examples/fit_draft.py [--steps 60 --batch 64 --draft 4 --vocab 4096 --hidden 128]

A stand-in for a drafter that reads the target's hidden states (random ones here,
and a random output layer as the target): the draft is an output layer of its own,
begun near zero.  Every step of the loop is a step of speculative decoding,
followed by what fits the draft to it:

  1. the draft proposes a token for each of K positions; ``verify`` accepts a
     prefix and draws the token after it;
  2. ``token_logprobs`` scores the emitted tokens under the target, with the
     entropy and the most likely alternatives (what a serving interface returns);
  3. ``distill`` compares the draft's rows with the target's at the positions the
     step has reached, and gives the gradient of the draft logits;
  4. the layer's gradients follow by two matrix products, ``clip_grads`` bounds
     their norm, and the layer takes a step.

``acceptance_rates`` shows the draft's acceptance probability rising.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_specv_gb300 as specv  # noqa: E402


def sample(logits, gen):
    """One token per row from softmax(logits), by the Gumbel-max trick."""
    u = torch.rand(logits.shape, generator=gen, device=logits.device).clamp_min_(1e-30)
    return (logits - torch.log(-torch.log(u))).argmax(-1).to(torch.int32)


def fit(steps=60, batch=64, draft=4, vocab=4096, hidden=128, lr=40.0, max_norm=0.05, seed=0,
        kind=specv.FORWARD_KL, report=print):
    """Runs the loop; returns a list of dicts, one per step."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    scale = 3.0 / hidden ** 0.5
    target_head = torch.randn((vocab, hidden), generator=gen, device=dev) * scale
    head = torch.randn((vocab, hidden), generator=gen, device=dev) * (0.1 * scale)
    bias = torch.zeros(vocab, device=dev)
    lam = torch.zeros(batch, device=dev)
    history = []
    for step in range(steps):
        h = torch.randn((batch, draft + 1, hidden), generator=gen, device=dev)
        target_logits = h @ target_head.T                       # [B][K+1][V]
        h_draft = h[:, :draft].reshape(batch * draft, hidden)
        draft_logits = (h_draft @ head.T + bias).view(batch, draft, vocab)
        proposed = sample(draft_logits, gen)
        tokens, n = specv.verify(target_logits, draft_logits, proposed,
                                 torch.rand((batch, draft), generator=gen, device=dev),
                                 torch.rand(batch, generator=gen, device=dev), lam)

        scored = specv.token_logprobs(target_logits, tokens, top_n=3)
        alpha = specv.acceptance_rates(target_logits, draft_logits, lam)

        # the positions that the step has reached: the accepted ones and the first rejected
        reached = torch.arange(draft, device=dev) <= n.unsqueeze(1)
        weight = reached.float() / reached.sum()
        loss, grad = specv.distill(target_logits, draft_logits, weight, kind=kind)
        grad = grad.view(batch * draft, vocab)
        grads = [grad.T @ h_draft, grad.sum(0)]
        norm = specv.clip_grads(grads, max_norm)
        head -= lr * grads[0]
        bias -= lr * grads[1]

        emitted = (tokens >= 0).sum()
        history.append(dict(step=step, loss=float(loss.sum()), alpha=float(alpha.mean()),
                            tokens_per_step=float(emitted) / batch, norm=float(norm),
                            logprob=float(scored.logprobs.sum() / emitted),
                            entropy=float(scored.entropy.sum() / emitted),
                            alternatives=scored.top_tokens[0, 0].tolist()))
        if report and (step % 10 == 0 or step == steps - 1):
            x = history[-1]
            report(f"step {step:4d}  loss {x['loss']:.4f}  acceptance {x['alpha']:.3f}  "
                   f"tokens per step {x['tokens_per_step']:.2f}  gradient norm {x['norm']:.3f}  "
                   f"ln p of emitted tokens {x['logprob']:.3f} (entropy {x['entropy']:.3f})")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--draft", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=128)
    ap.add_argument("--reverse", action="store_true", help="KL(draft || target)")
    a = ap.parse_args()
    fit(a.steps, a.batch, a.draft, a.vocab, a.hidden,
        kind=specv.REVERSE_KL if a.reverse else specv.FORWARD_KL)
