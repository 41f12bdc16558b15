"""Binding of the rotary calls (include/kvq.h, "Rotary positions").

A model's frequencies are made once, a step's angles once for all layers, and
the layers turn their queries and keys by them::

    turns = kvq_rotary_turns(rotary_dim=128, base=500000.0)
    angles = kvq_rotary_angles(positions, turns)             # once a step
    q = kvq_rotate(q, angles)                                # every layer
    cache.append(k, v, slots, angles, q=q, q_out=q)          # or turned on the way

positions come from kvq_paged_plan.  The calls run on the tensors' device, on
torch's current stream of it unless `stream` is given (a stream or its
address), and can be captured into CUDA graphs.  Nothing here has a gradient.
"""
from __future__ import annotations

import ctypes

import torch

from . import kvq
from .kvq import KVQ_ERR_INVALID_ARG, KVQ_ERR_UNSUPPORTED, KvqError
from .paged import _paged_bind

_angles = _paged_bind.angles
_rotate = _paged_bind.rotate


def kvq_rotary_turns(rotary_dim: int, base: float = 10000.0, factor: float = 1.0,
                     original_len: float = 0.0, low: float = 1.0, high: float = 32.0,
                     device="cuda"):
    """Frequencies base^(-2 i / rotary_dim) as int64 parts of a turn, units of
    2^-64, [rotary_dim / 2], within 2^-51 of a turn (float64's roundings).

    factor > 1 slows the pairs down for longer contexts: all of them where
    original_len is 0, else those that make few turns in original_len positions
    (all the way at `low` turns, not at all from `high` on)."""
    try:
        n = int(rotary_dim)
        whole = n == rotary_dim
    except (TypeError, ValueError, OverflowError):
        whole = False
    if not whole or n < 2 or n % 2:
        raise KvqError(KVQ_ERR_INVALID_ARG, "kvq_rotary_turns: rotary_dim must be even and positive")
    if n > 256:
        raise KvqError(KVQ_ERR_UNSUPPORTED, "kvq_rotary_turns: rotary_dim must be at most 256")
    turns = (ctypes.c_int64 * (n // 2))()
    kvq._check(kvq._lib.kvq_rotary_turns(turns, n, float(base), float(factor), float(original_len),
                                         float(low), float(high)), "kvq_rotary_turns")
    return torch.tensor(list(turns), dtype=torch.int64, device=device)


def kvq_rotary_angles(positions, turns, magnitude: float = 1.0, out=None, stream=None):
    """Cosines and sines, times magnitude, of the tokens' angles: fp32
    [tokens][rotary_dim / 2][2].  positions: int32 [tokens], any values; turns:
    kvq_rotary_turns."""
    return _angles(positions, turns, magnitude, out, stream)


def kvq_rotate(x, angles, interleaved: bool = False, out=None, stream=None):
    """x (fp16 or bf16 [tokens][heads][head_dim], any token stride that is a
    multiple of 8) with the first rotary_dim channels of every head turned by
    its token's angles: channels (i, i + rotary_dim / 2), or (2 i, 2 i + 1) where
    interleaved.  Returns out, which may be x itself, or a new tensor."""
    return _rotate(x, angles, interleaved, out, stream)
