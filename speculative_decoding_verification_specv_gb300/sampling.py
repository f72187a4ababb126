"""Drawing tokens from logits under sampling parameters, and the filtered logits that
the verify step takes for the same distribution.

As in the rest of the binding, tensors are checked, pointers and the current stream
passed on, and status codes turned into exceptions; every kernel runs in
``libspecv.so``.  Logits may be views, as for token_logprobs.
"""
from __future__ import annotations

import struct
from typing import NamedTuple

import torch

from . import BF16, F32, _check, _dtype_code
from .scoring import _elsewhere, _entry, _fit, _rows, _stream

_Tensor, _empty, _f32, _i32 = torch.Tensor, torch.empty, torch.float32, torch.int32
_written = torch.autograd.graph.increment_version  # a graph that saved the tensor sees it
# specv_sampling: four pointers and, for those that are NULL, the values for all rows
_pack = struct.Struct("PPPPfiff").pack


class SampledTokens(NamedTuple):
    """Of every row: the token, ln of its probability among the kept entries, and the
    log-normaliser of the kept entries' logits over the temperature."""
    tokens: torch.Tensor
    logprobs: torch.Tensor
    logsumexp: torch.Tensor


def _params(temperature, top_k, top_p, min_p, lead, dev) -> bytes:
    at = [0, 0, 0, 0]
    if isinstance(temperature, _Tensor):
        _fit(temperature, "temperature", _f32, lead, dev)
        at[0], temperature = temperature.data_ptr(), 1.0
    else:
        temperature = 1.0 if temperature is None else float(temperature)
        if not 0.0 <= temperature <= 3.4e38:
            raise ValueError("temperature must be >= 0 and finite")
    if isinstance(top_k, _Tensor):
        _fit(top_k, "top_k", _i32, lead, dev)
        at[1], top_k = top_k.data_ptr(), 0
    else:
        top_k = 0 if top_k is None else int(top_k)
        top_k = min(max(top_k, 0), 2**31 - 1)  # below 1 and from V on: off
    if isinstance(top_p, _Tensor):
        _fit(top_p, "top_p", _f32, lead, dev)
        at[2], top_p = top_p.data_ptr(), 1.0
    else:
        top_p = 1.0 if top_p is None else float(top_p)
        if not top_p >= 0.0:
            raise ValueError("top_p must be >= 0")
        top_p = min(top_p, 2.0)  # from 1 on: off
    if isinstance(min_p, _Tensor):
        _fit(min_p, "min_p", _f32, lead, dev)
        at[3], min_p = min_p.data_ptr(), 0.0
    else:
        min_p = 0.0 if min_p is None else float(min_p)
        if not 0.0 <= min_p <= 1.0:
            raise ValueError("min_p must be in 0..1")
    return _pack(*at, temperature, top_k, top_p, min_p)


def _out_code(out, name, logits, dev) -> int:
    if not isinstance(out, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if out.dtype is not _f32 and out.dtype is not logits.dtype:
        raise TypeError(f"{name} must be float32 or {logits.dtype}, got {out.dtype}")
    _fit(out, name, out.dtype, logits.shape, dev)
    return F32 if out.dtype is _f32 else BF16


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None,
                  out_filtered=None, stream=None) -> SampledTokens:
    """One token per row of logits, by inverse CDF from the uniform u.

    logits [B][N][V] or [N][V] (float32 or bfloat16; the last dimension contiguous,
    the others of any strides), u float32 of the leading shape, in [0, 1].
    temperature (0: greedy), top_k (below 1: off), top_p (from 1 on: off) and min_p
    (0: off) are numbers for all rows or contiguous tensors of the leading shape,
    float32 (top_k: int32), as a batch of requests has them; None leaves each out.
    Entries are ordered by falling logits, equal ones by rising index: top_k keeps the
    first, top_p the fewest first that hold that share of what top_k keeps, min_p
    those of at least min_p times the largest probability.  The token is the first
    kept index whose running sum exceeds u times the kept sum (at 1 the last kept one);
    weights are fp32 exponentials, the largest 1, each rounded to 2^-44 (V above 2^18: to
    2^-62 times the next power of two) for the sums that decide: below half of that it
    counts as none.

    With ``out_filtered`` (contiguous, of the logits' shape, float32 or the logits'
    type; may be the logits themselves) the filtered rows are written as well, as
    filter_logits returns them.

    Masked (-inf) entries are never drawn; a row that masks every entry gives -1, with a
    log probability of 0.  A row with a NaN or +inf, a u outside [0, 1] or a row's
    parameter outside its range gives -1 and NaN.  Asynchronous on ``stream`` (default:
    the current stream), on which the results are allocated.
    """
    B, N, V, sb, sn = _rows(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    code = _dtype_code(logits)
    _fit(u, "u", _f32, lead, dev)
    params = _params(temperature, top_k, top_p, min_p, lead, dev)
    out_code = code if out_filtered is None else _out_code(out_filtered, "out_filtered", logits, dev)
    there = _elsewhere(stream, dev)
    if there is not None:
        with there:
            return sample_tokens(logits, u, temperature, top_k, top_p, min_p, out_filtered)
    tokens = _empty(lead, dtype=_i32, device=dev)
    logprobs = _empty(lead, dtype=_f32, device=dev)
    lse = _empty(lead, dtype=_f32, device=dev)
    st = _entry("specv_sample_tokens")(
        logits.data_ptr(), u.data_ptr(), params, B, N, V, sb, sn, code, tokens.data_ptr(),
        logprobs.data_ptr(), lse.data_ptr(),
        None if out_filtered is None else out_filtered.data_ptr(), out_code, _stream(dev))
    if st:
        _check(st, "specv_sample_tokens")
    if out_filtered is not None:
        _written(out_filtered)
    return SampledTokens(tokens, logprobs, lse)


def filter_logits(logits, temperature=None, top_k=None, top_p=None, min_p=None, out=None,
                  dtype=None, stream=None) -> torch.Tensor:
    """Rows of logits over their temperature, -inf where an entry is not kept.

    logits and parameters as for sample_tokens.  The softmax of a filtered row is the
    distribution that sample_tokens draws from, so ``verify`` on filtered target and
    draft rows, with tokens drawn from the draft's, keeps the target's distribution
    under its sampling parameters.  Returns a contiguous tensor of the logits' shape:
    ``out`` if given (float32 or the logits' type; may be the logits themselves), else a
    new one of ``dtype`` (default: the logits').  In bfloat16 a temperature other than
    1 rounds the values, and with them the distribution; float32 rows hold it to
    rounding.  A temperature of 0 gives 0 at the largest entry.  Rows that mask every
    entry stay so; rows with a NaN or +inf, or with a parameter outside its range, become
    NaN.
    """
    B, N, V, sb, sn = _rows(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    code = _dtype_code(logits)
    params = _params(temperature, top_k, top_p, min_p, lead, dev)
    if out is not None:
        out_code = _out_code(out, "out", logits, dev)
        if dtype is not None and dtype is not out.dtype:
            raise TypeError(f"out must be {dtype}, got {out.dtype}")
    else:
        dtype = logits.dtype if dtype is None else dtype
        if dtype is not _f32 and dtype is not logits.dtype:
            raise TypeError(f"dtype must be torch.float32 or {logits.dtype}, got {dtype}")
        out_code = F32 if dtype is _f32 else BF16
    there = _elsewhere(stream, dev)
    if there is not None:
        with there:
            return filter_logits(logits, temperature, top_k, top_p, min_p, out, dtype)
    given = out is not None
    if not given:
        out = _empty(logits.shape, dtype=dtype, device=dev)
    st = _entry("specv_filter_logits")(logits.data_ptr(), params, B, N, V, sb, sn, code,
                                       out.data_ptr(), out_code, _stream(dev))
    if st:
        _check(st, "specv_filter_logits")
    if given:
        _written(out)
    return out
