"""Operators on the logits that a verify step leaves behind: log probabilities of
the emitted tokens (and their gradient), the loss that fits a draft to its
target, and clipping of the draft's gradients.

As in the rest of the binding, tensors are checked, pointers and the current
stream passed on, and status codes turned into exceptions; every kernel runs in
``libspecv.so``.  Logits may be views: the last dimension is contiguous, the
others have any strides (rows of a padded vocabulary, ``target_logits[:, :K]``).
"""
from __future__ import annotations

from array import array
from operator import attrgetter
from typing import NamedTuple, Optional

import torch

from . import BF16, F32, _check, _dtype_code, _require, load

FORWARD_KL = 0  # KL(target || draft)
REVERSE_KL = 1  # KL(draft || target)
MAX_TOP = 32


class TokenLogprobs(NamedTuple):
    """Of every row: ln p(token), the entropy, (max, ln sum exp(z - max)), and the
    top_n most likely tokens with their log probabilities (None when top_n is 0)."""
    logprobs: torch.Tensor
    entropy: torch.Tensor
    stats: torch.Tensor
    top_tokens: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


# These calls are short enough on the GPU that the host's part of one counts: entry
# points are looked up once, a tensor that fits is passed with a single test, and the
# stream's handle is asked for without building a Stream object.
_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_Tensor, _empty, _f32, _i32 = torch.Tensor, torch.empty, torch.float32, torch.int32
_entries: dict = {}


def _entry(name: str):
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(load(), name)
    return fn


def _elsewhere(stream, dev):
    """The context that a call on tensors of ``dev`` is to be made in, or None.

    Where ``dev`` is not current it becomes so (the library launches on the current
    device, and takes its scratch there).  A given stream becomes the current one, so
    that the results are allocated on it too: memory of another stream could still be in
    use there when the kernel writes it, or be given away there before the kernel has."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream must be of {dev}, got {stream.device}")
        return torch.cuda.stream(stream)
    return None if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _fit(t, name: str, dtype, shape, dev):
    """A contiguous tensor of this type, shape and device, else the error that says why."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == dev and t.is_contiguous()):
        _require(t, name, dtype, shape, dev)


def _rows(t: torch.Tensor, name: str):
    """(B, N, V, stride_b, stride_n) of logits [B][N][V] or [N][V] on the GPU."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() == 3:
        (B, N, V), (sb, sn, sv) = t.shape, t.stride()
    elif t.dim() == 2:
        (N, V), (sn, sv) = t.shape, t.stride()
        B, sb = 1, 0
    else:
        raise ValueError(f"{name} must be [B][N][V] or [N][V]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the kernels run only on the GPU)")
    if sv != 1 and V > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return B, N, V, sb, sn


def token_logprobs(logits, tokens, top_n: int = 0, stream=None) -> TokenLogprobs:
    """Log probabilities of given tokens, with entropy and top alternatives.

    logits [B][N][V] or [N][V] (float32 or bfloat16; strides as above), tokens
    int32 of the leading shape: ``verify``'s out_tokens, for instance.  A token of
    -1 is no token: its row is not read, its log probability and entropy are 0 and
    its alternatives (-1, -inf).  Alternatives are ordered by value, ties by the
    lower token; masked (-inf) entries are none.  Rows with a NaN or +inf, or with
    a token outside [0, V), give NaN; rows that mask every entry a log probability
    of -inf and an entropy of 0.  Asynchronous on ``stream`` (default: the current
    stream), on which the results are allocated.  No autograd graph is recorded: token_logprobs_backward is the gradient.
    """
    B, N, V, sb, sn = _rows(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    code = _dtype_code(logits)
    _fit(tokens, "tokens", _i32, lead, dev)
    n = int(top_n)
    if not 0 <= n <= MAX_TOP:
        raise ValueError(f"top_n must be in 0..{MAX_TOP}")
    there = _elsewhere(stream, dev)
    if there is not None:
        with there:
            return token_logprobs(logits, tokens, n)
    logprobs = _empty(lead, dtype=_f32, device=dev)
    entropy = _empty(lead, dtype=_f32, device=dev)
    stats = _empty((*lead, 2), dtype=_f32, device=dev)
    top_t = top_l = None
    if n:
        top_t = _empty((*lead, n), dtype=_i32, device=dev)
        top_l = _empty((*lead, n), dtype=_f32, device=dev)
    st = _entry("specv_token_logprobs")(
        logits.data_ptr(), tokens.data_ptr(), B, N, V, sb, sn, code, n, logprobs.data_ptr(),
        entropy.data_ptr(), stats.data_ptr(), top_t.data_ptr() if n else None,
        top_l.data_ptr() if n else None, _stream(dev))
    if st:
        _check(st, "specv_token_logprobs")
    return TokenLogprobs(logprobs, entropy, stats, top_t, top_l)


def token_logprobs_backward(logits, tokens, stats, entropy, grad_logprobs, grad_entropy=None,
                            out=None, stream=None) -> torch.Tensor:
    """The gradient with respect to the logits of token_logprobs, from the
    gradients of its log probabilities and (optionally) entropies.

    logits and tokens as in the forward call, stats and entropy what it returned.
    Returns a contiguous tensor of the logits' shape and type (``out`` if given,
    which may be the logits themselves).  Rows without a token, and rows that
    mask every entry, get zeros.
    """
    B, N, V, sb, sn = _rows(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    code = _dtype_code(logits)
    _fit(tokens, "tokens", _i32, lead, dev)
    _fit(stats, "stats", _f32, (*lead, 2), dev)
    _fit(entropy, "entropy", _f32, lead, dev)
    _fit(grad_logprobs, "grad_logprobs", _f32, lead, dev)
    if grad_entropy is not None:
        _fit(grad_entropy, "grad_entropy", _f32, lead, dev)
    if out is not None:
        _fit(out, "out", logits.dtype, logits.shape, dev)
    there = _elsewhere(stream, dev)
    if there is not None:
        with there:
            return token_logprobs_backward(logits, tokens, stats, entropy, grad_logprobs,
                                           grad_entropy, out)
    if out is None:
        out = _empty(logits.shape, dtype=logits.dtype, device=dev)
    st = _entry("specv_token_logprobs_backward")(
        logits.data_ptr(), tokens.data_ptr(), stats.data_ptr(), entropy.data_ptr(),
        grad_logprobs.data_ptr(), None if grad_entropy is None else grad_entropy.data_ptr(), B, N,
        V, sb, sn, code, out.data_ptr(), _stream(dev))
    if st:
        _check(st, "specv_token_logprobs_backward")
    return out


def distill(target_logits, draft_logits, weight=None, kind: int = FORWARD_KL, need_grad: bool = True,
            out_grad=None, stream=None):
    """The divergence of the draft's rows from the target's, and its gradient with
    respect to the draft logits: (loss [B][K] float32, grad [B][K][V]).

    target_logits [B][K][V] or [B][K+1][V] (the verify step's, whose last row is
    not read), draft_logits [B][K][V] of the same type, weight float32 [B][K] or
    None (ones).  loss is weight * KL, kind FORWARD_KL (target over draft) or
    REVERSE_KL (draft over target); grad is the gradient of loss.sum(), in the
    logits' type, contiguous (``out_grad`` if given, which may be draft_logits
    itself), or None without ``need_grad``.  Positions of weight 0 are not read.
    """
    B, K, V, dsb, dsk = _rows(draft_logits, "draft_logits")
    Bt, Kt, Vt, tsb, tsk = _rows(target_logits, "target_logits")
    if draft_logits.dim() != 3 or target_logits.dim() != 3:
        raise ValueError("target_logits and draft_logits must be [B][K][V]")
    if Bt != B or Vt != V or Kt not in (K, K + 1):
        raise ValueError(f"target_logits must be [{B}][{K} or {K + 1}][{V}], got "
                         f"{tuple(target_logits.shape)}")
    dev = draft_logits.device
    if target_logits.device != dev:
        raise ValueError(f"target_logits must be on {dev}, got {target_logits.device}")
    code = _dtype_code(draft_logits)
    if target_logits.dtype != draft_logits.dtype:
        raise TypeError(f"target_logits must be {draft_logits.dtype}, got {target_logits.dtype}")
    if weight is not None:
        _fit(weight, "weight", torch.float32, (B, K), dev)
    if kind not in (FORWARD_KL, REVERSE_KL):
        raise ValueError("kind must be FORWARD_KL (0) or REVERSE_KL (1)")
    if out_grad is not None:
        _fit(out_grad, "out_grad", draft_logits.dtype, (B, K, V), dev)
    there = _elsewhere(stream, dev)
    if there is not None:
        with there:
            return distill(target_logits, draft_logits, weight, kind, need_grad, out_grad)
    loss = _empty((B, K), dtype=_f32, device=dev)
    if out_grad is None and need_grad:
        out_grad = _empty((B, K, V), dtype=draft_logits.dtype, device=dev)
    st = _entry("specv_distill")(
        target_logits.data_ptr(), draft_logits.data_ptr(),
        None if weight is None else weight.data_ptr(), B, K, V, tsb, tsk, dsb, dsk, code,
        int(kind), loss.data_ptr(), None if out_grad is None else out_grad.data_ptr(),
        _stream(dev))
    if st:
        _check(st, "specv_distill")
    return loss, out_grad


def clip_grads(grads, max_norm: float, out=None, stream=None) -> torch.Tensor:
    """Clip gradients to a largest 2-norm over all of them; returns the norm before
    clipping (float32, no host synchronisation).

    grads: float32 and bfloat16 CUDA tensors, contiguous, of any shapes (empty
    ones too), none twice.  Clipped in place, or into ``out`` (one tensor for each
    gradient, of its size and type; the gradient itself may stand there).  Values
    are scaled by min(1, max_norm / (norm + 1e-6)); a norm that is not finite
    leaves them as they are.  max_norm = inf only measures.
    """
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError(f"out must hold {len(grads)} tensors, got {len(out)}")
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError("max_norm must be >= 0")
    at, counts, codes = _table(grads, "gradient")
    if grads:
        dev = grads[0].device
    elif stream is not None:
        dev = stream.device
    else:
        dev = torch.device("cuda", torch.cuda.current_device())
    if out is grads:
        to = at
    else:
        to, sizes, types = _table(out, "out")
        if sizes != counts or types != codes or (out and out[0].device != dev):
            raise ValueError("out must match the gradients in type, size and device")
    live = [p for p, n in zip(at, counts) if n]
    if len(set(live)) != len(live):
        raise ValueError("a gradient is listed twice")
    there = _elsewhere(stream, dev)
    if there is not None:
        with there:
            return clip_grads(grads, max_norm, None if out is grads else out)
    table = array("q", bytes(32 * len(grads)))
    table[0::4], table[1::4] = array("q", at), array("q", to)
    table[2::4], table[3::4] = array("q", counts), array("q", codes)
    norm = _empty((), dtype=_f32, device=dev)
    st = _entry("specv_clip_grads")(table.buffer_info()[0] if grads else None, len(grads), max_norm,
                                    norm.data_ptr(), _stream(dev))
    if st:
        _check(st, "specv_clip_grads")
    return norm


def _table(tensors, name: str):
    """(addresses, sizes, type codes) of contiguous CUDA tensors of one device."""
    at = list(map(torch.Tensor.data_ptr, tensors))
    devices = set(map(torch.Tensor.get_device, tensors))  # -1: not a CUDA device
    if len(devices) > 1 or -1 in devices:
        raise ValueError("gradients must be CUDA tensors of one device")
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError(f"every {name} must be contiguous")
    try:
        codes = [_CODES[t] for t in map(attrgetter("dtype"), tensors)]
    except KeyError as e:
        raise TypeError(f"gradients must be float32 or bfloat16, got {e.args[0]}") from None
    return at, list(map(torch.Tensor.numel, tensors)), codes
