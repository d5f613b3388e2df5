"""Plain fp64 definitions of the paged key/value cache operators.

TEST INFRASTRUCTURE ONLY, like :mod:`oracle.chain`: evaluated in float64 from the
storage-dtype inputs, one sequence and one head at a time.  Pinned by
``tests/test_kv_host.py`` against closed forms and torch's float64 attention.
"""
from __future__ import annotations

import numpy as np

from .chain import to64


def rotate(x, cos, sin, pairing: str) -> np.ndarray:
    """x [..., d] with its first 2 * len(cos) dimensions rotated by the angles whose
    cosines and sines are given ([..., rotary_dim / 2], broadcast over heads)."""
    x, cos, sin = to64(x).copy(), to64(cos), to64(sin)
    h = cos.shape[-1]
    lo, hi = (np.arange(h), np.arange(h) + h) if pairing == "half" else (2 * np.arange(h), 2 * np.arange(h) + 1)
    a, b = x[..., lo], x[..., hi]
    x[..., lo], x[..., hi] = a * cos - b * sin, b * cos + a * sin
    return x


def visible(pos: int, count: int, window: int, sinks: int, prefix: int = 0) -> np.ndarray:
    """Which of the prefix + count keys of a sequence its token at position pos sees."""
    j = np.arange(count)
    own = (j <= pos) if window <= 0 else (j <= pos) & ((j > pos - window) | (j < sinks))
    return np.concatenate([np.ones(prefix, dtype=bool), own])


def attend(q, k, v, seen, scale: float):
    """One query and head over keys [n, d]: (softmax(scale q.k) v, log-sum-exp, sum of weight * |v|).
    Hidden keys are left out, whatever they hold; without a visible key: zeros, -inf, zeros."""
    k, v = to64(k)[seen], to64(v)[seen]
    if len(k) == 0:
        return np.zeros(q.shape[-1]), -np.inf, np.zeros(q.shape[-1])
    s = (k @ to64(q)) * scale
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    return p @ v / total, m + np.log(total), p @ np.abs(v) / total
