"""The optimizer's step on the draft's weights: AdamW over many tensors in one call,
clipped by the norm that clip_grads has measured, with states in 32 or in 8 bits.

As in the rest of the binding, tensors are checked, pointers and the current stream
passed on, and status codes turned into exceptions; every kernel runs in
``libspecv.so``.
"""
from __future__ import annotations

import math
import struct
from array import array
from operator import attrgetter
from typing import List, NamedTuple, Optional

import torch

from . import _check
from .scoring import _CODES, _elsewhere, _entry, _stream

_Tensor, _f32 = torch.Tensor, torch.float32
_f8 = torch.float8_e4m3fn
BLOCK = 256  # entries of an 8-bit state that share a scale
# specv_adamw_config
_pack = struct.Struct("qqddddPPPfIQ").pack
_WORDS = 10  # of specv_adamw_tensor
_EITHER = (torch.float32, torch.bfloat16)
_MOST = torch.finfo(torch.float32).max
_dtype_of, _get_device = attrgetter("dtype"), _Tensor.get_device
_written = torch.autograd.graph.increment_version


class AdamWState(NamedTuple):
    """The state of adamw_step, one entry for each weight: the averages of the gradient and
    of its square (32 bits: float32; 8 bits: float8_e4m3fn values m / s_m and
    sqrt(v) / s_r), the scales (s_m, s_r) of every 256 entries (None in 32 bits), and the
    float32 masters (None, or None for a weight without one)."""
    exp_avg: List[torch.Tensor]
    exp_avg_sq: List[torch.Tensor]
    scales: Optional[List[torch.Tensor]]
    masters: Optional[List[Optional[torch.Tensor]]]


def adamw_state(params, bits: int = 32, masters: bool = False) -> AdamWState:
    """The state before the first step: zeros, and with ``masters`` a float32 copy of every
    bfloat16 weight.  bits: 32, or 8 (2 bytes and a 32nd of a byte for each entry)."""
    params = list(params)
    if bits not in (8, 32):
        raise ValueError("bits must be 32 or 8")
    kind = _f32 if bits == 32 else _f8
    avg = [torch.zeros(p.shape, dtype=kind, device=p.device) for p in params]
    sq = [torch.zeros(p.shape, dtype=kind, device=p.device) for p in params]
    scales = None if bits == 32 else [
        torch.zeros((-(-p.numel() // BLOCK), 2), dtype=_f32, device=p.device) for p in params]
    copies = [None if p.dtype is _f32 else p.detach().float() for p in params] if masters else None
    return AdamWState(avg, sq, scales, copies)


def _why(lists, n, dev, counts):
    """The error that says which of the lists does not fit."""
    for name, tensors, sizes, kind in lists:
        if len(tensors) != n[name]:
            raise ValueError(f"{name} must hold {n[name]} tensors, got {len(tensors)}")
        for t, c in zip(tensors, sizes):
            if not isinstance(t, _Tensor):
                raise TypeError(f"{name} must hold tensors, got {type(t).__name__}")
            if t.device != dev:
                raise ValueError(f"every tensor of {name} must be on {dev}, got {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"every tensor of {name} must be contiguous")
            if t.numel() != c:
                raise ValueError(f"{name} must match the weights in size: {c}, got {t.numel()}")
            if t.dtype not in kind:
                raise TypeError(f"{name} must be {' or '.join(map(str, kind))}, got {t.dtype}")
    raise ValueError("the tensors do not fit one another")


def _scalar(x, name: str, kind, dev):
    if x.dtype is not kind or x.numel() != 1 or x.device != dev:
        raise ValueError(f"{name} must be a {kind} tensor of one element on {dev}")
    return x.data_ptr()


def adamw_step(params, grads, state, step, lr, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay=0.0, norm=None, max_norm: float = math.inf, seed: int = 0,
               stream=None) -> None:
    """One AdamW step over many tensors, in place.

    params and grads: float32 and bfloat16 CUDA tensors of one device, contiguous, of any
    shapes (empty ones too), none twice; a gradient has its weight's shape (or the same
    entries in one dimension, as the state may) and either type.  state: an AdamWState (adamw_state makes the first), or its four fields.
    step: the step's number, from 1 on; lr: the learning rate.  Either may be a CUDA
    tensor of one element (int32, float32), which a captured graph reads anew at each
    replay.  eps: 0, or a normal float32 number.  weight_decay: a number, or one for each
    weight.

    norm: the gradients' norm as clip_grads returns it; they are then scaled by
    min(1, max_norm / (norm + 1e-6)) as they are read (and left as they are: measure with
    ``clip_grads(grads, math.inf)``).  A norm that is not finite leaves weights and state
    as they are.

    As after any step in place, autograd refuses to go back through a graph that saved the
    weights before it.  (A replayed CUDA graph writes them unseen.)

    8-bit states are rounded at random, reproducibly: by ``seed``, the step, the tensor's
    place in the list and the entry's place in the tensor.
    """
    params, grads = list(params), list(grads)
    exp_avg, exp_avg_sq, scales, masters = state
    n = len(params)
    try:
        counts = list(map(_Tensor.numel, params))
    except TypeError:
        raise TypeError("params must hold tensors") from None
    if n:
        dev = params[0].device
        if dev.type != "cuda":
            raise ValueError("params must be CUDA tensors (the kernels run only on the GPU)")
    elif stream is not None:
        dev = stream.device
    else:
        dev = torch.device("cuda", torch.cuda.current_device())
    bits = 32 if scales is None else 8
    # A call is short on the GPU: all tensors are looked at together, in a few passes.
    exp_avg, exp_avg_sq = list(exp_avg), list(exp_avg_sq)
    kind = (_f32,) if bits == 32 else (_f8,)
    lists = [("params", params, counts, _EITHER), ("grads", grads, counts, _EITHER),
             ("exp_avg", exp_avg, counts, kind), ("exp_avg_sq", exp_avg_sq, counts, kind)]
    lengths = dict.fromkeys(("params", "grads", "exp_avg", "exp_avg_sq"), n)
    if bits == 8:
        scales = list(scales)
        lists.append(("scales", scales, [2 * (-(-c // BLOCK)) for c in counts], (_f32,)))
        lengths["scales"] = n
    some = []
    if masters is not None:
        if len(masters) != n:
            raise ValueError(f"masters must hold {n} entries, got {len(masters)}")
        some = [i for i, w in enumerate(masters) if w is not None]
        lists.append(("masters", [masters[i] for i in some], [counts[i] for i in some], (_f32,)))
        lengths["masters"] = len(some)
    every, sizes = [], []
    for _, tensors, c, _ in lists:
        every += tensors
        sizes += c
    types = None
    try:
        if (len(every) == len(sizes) and all(map(_Tensor.is_contiguous, every))
                and set(map(_get_device, every)) <= {dev.index}
                and list(map(_Tensor.numel, every)) == sizes):
            types = list(map(_dtype_of, every))
            codes = list(map(_CODES.get, types[:2 * n]))
            if (None in codes or set(types[2 * n:4 * n]) - set(kind)
                    or set(types[4 * n:]) - {_f32}):
                types = None
    except TypeError:  # not a tensor
        pass
    if types is None or any(len(t) != lengths[name] for name, t, _, _ in lists):
        _why(lists, lengths, dev, counts)
    # Of two matrices of one size, one may be the other's transpose: shapes have to agree.
    # (Flat ones may stand for any shape.)
    deep = [i for i, d in enumerate(map(_Tensor.dim, params)) if d > 1]
    if deep:
        for name, tensors, of in (("grads", grads, deep), ("exp_avg", exp_avg, deep),
                                  ("exp_avg_sq", exp_avg_sq, deep),
                                  ("masters", masters, [i for i in some if params[i].dim() > 1])):
            for i in of:
                if tensors[i].shape != params[i].shape and tensors[i].dim() > 1:
                    raise ValueError(f"{name} must match the weights in shape: "
                                     f"{tuple(params[i].shape)}, got {tuple(tensors[i].shape)}")
    at = list(map(_Tensor.data_ptr, every))
    # (gradients are only read: one may serve several weights)
    live = at[:n] + at[2 * n:]
    if len(set(live)) != len(live):  # (empty tensors may share an address)
        live = [p for p, c in zip(live, counts + sizes[2 * n:]) if c]
        if len(set(live)) != len(live):
            raise ValueError("a weight, a state or a master is listed twice")
    table = array("q", bytes(8 * _WORDS * n))
    for k in range(5 if bits == 8 else 4):
        table[k::_WORDS] = array("q", at[k * n:(k + 1) * n])
    for i, p in zip(some, at[len(at) - len(some):]):
        table[_WORDS * i + 5] = p
    table[6::_WORDS] = array("q", counts)
    table[7::_WORDS], table[8::_WORDS] = array("q", codes[:n]), array("q", codes[n:])
    if isinstance(weight_decay, (int, float)):
        decay = array("d", [weight_decay]) * n
    else:
        decay = array("d", weight_decay)
        if len(decay) != n:
            raise ValueError(f"weight_decay must be a number or {n} of them, got {len(decay)}")
    table[9::_WORDS] = array("q", decay.tobytes())
    if decay and not all(0.0 <= x < math.inf for x in set(decay)):
        raise ValueError("weight_decay must be >= 0 and finite")
    step_at = lr_at = norm_at = 0
    if isinstance(step, _Tensor):
        step_at, step = _scalar(step, "step", torch.int32, dev), 0
    else:
        step = int(step)
        if step < 1:
            raise ValueError("step must be >= 1")
    if isinstance(lr, _Tensor):
        lr_at, lr = _scalar(lr, "lr", _f32, dev), 0.0
    else:
        lr = float(lr)
        if not 0.0 <= lr < math.inf:
            raise ValueError("lr must be >= 0 and finite")
    b1, b2 = float(betas[0]), float(betas[1])
    if not (0.0 <= b1 < 1.0 and 0.0 <= b2 < 1.0):
        raise ValueError("betas must be in [0, 1)")
    eps = float(eps)
    if eps != 0.0 and not 2.0**-126 <= eps < math.inf:  # (flushed to 0 below)
        raise ValueError("eps must be 0 or a normal float32 number")
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError("max_norm must be >= 0")
    if max_norm > _MOST:  # no norm in float32 exceeds it
        max_norm = math.inf
    if norm is not None:
        norm_at = _scalar(norm, "norm", _f32, dev)
    elif max_norm != math.inf:
        raise ValueError("max_norm needs the gradients' norm")
    config = _pack(bits, step, lr, b1, b2, eps, step_at, lr_at, norm_at, max_norm, 0,
                   seed & 0xFFFFFFFFFFFFFFFF)
    there = _elsewhere(stream, dev)
    if there is None:
        st = _entry("specv_adamw_step")(table.buffer_info()[0] if n else None, n, config,
                                        _stream(dev))
    else:
        with there:
            st = _entry("specv_adamw_step")(table.buffer_info()[0] if n else None, n, config,
                                            _stream(dev))
    if st:
        _check(st, "specv_adamw_step")
    # a graph that saved a weight sees that it was written
    _written(params if not some else params + [masters[i] for i in some])
