"""Plain fp64 definitions of the key/value cache held in 4 bits.

TEST INFRASTRUCTURE ONLY, like :mod:`oracle.kv`: the format of ``include/cs_kv4.h``, by
search through all 248 scales.  Pinned by ``tests/test_kv4_host.py``.
"""
from __future__ import annotations

import numpy as np

from .chain import to64

GROUP = 32
NAN_BYTE = 0xFF
_E, _M = np.arange(256) // 8, np.arange(256) % 8
SCALES = np.where(_E == 0, _M / 8 * 2.0 ** -14, (1 + _M / 8) * 2.0 ** (_E - 15.0))
SCALES[0xF8:] = np.nan
FINITE = SCALES[:0xF8]


def quantise(x):
    """(codes c, scale bytes) of x [..., d]: int8 [..., d] and uint8 [..., d / 32]."""
    x = to64(x)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.abs(g).max(-1)
    hi = np.clip(np.searchsorted(7 * FINITE, amax), 1, len(FINITE) - 1)  # 7 FINITE[hi - 1] < amax <= 7 FINITE[hi]
    below, above = amax - 7 * FINITE[hi - 1], 7 * FINITE[hi] - amax
    byte = np.where((below > above) | ((below == above) & (hi % 2 == 0)), hi, hi - 1)
    s = FINITE[byte][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(s > 0, np.clip(np.rint(g / s), -7, 7), 0.0)
    byte = np.where(bad, NAN_BYTE, byte).astype(np.uint8)
    return c.astype(np.int8).reshape(x.shape), byte


def values(c, byte):
    """What codes and scale bytes stand for, float64."""
    c = np.asarray(c, dtype=np.float64)
    return (c.reshape(*c.shape[:-1], -1, GROUP) * SCALES[byte][..., None]).reshape(c.shape)


def held(x):
    return values(*quantise(x))


def pack(c):
    """Bytes [..., d / 2] of codes [..., d]: value 2 j of 8 at bit 4 j of a 32-bit word, value 2 j + 1 at bit 16 + 4 j."""
    u = (np.asarray(c).astype(np.int64) + 8).reshape(*np.shape(c)[:-1], -1, 8)
    word = sum(u[..., v] << (4 * (v // 2) + 16 * (v % 2)) for v in range(8))
    return word.astype("<u4").view(np.uint8).reshape(*np.shape(c)[:-1], -1)


def unpack(b):
    """Codes [..., d] of bytes [..., d / 2]."""
    word = np.ascontiguousarray(b).view("<u4").astype(np.int64)
    c = np.stack([(word >> (4 * (v // 2) + 16 * (v % 2)) & 15) - 8 for v in range(8)], -1)
    return c.reshape(*c.shape[:-2], -1).astype(np.int8)
