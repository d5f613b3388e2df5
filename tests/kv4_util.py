"""Batches of :mod:`kv_util` over a cache in 4 bits."""
from __future__ import annotations

import numpy as np
import torch

from kv_util import Batch
from oracle import kv4 as o4


def parts(cache, layout, seed=0):
    """(codes, scales) of a 16-bit cache; groups that hold a value that is not finite get scale 0xFF and any codes."""
    c, byte = o4.quantise(cache)
    r = np.random.default_rng(seed)
    bad = np.repeat(byte == o4.NAN_BYTE, o4.GROUP, axis=-1)
    c = np.where(bad, r.integers(-7, 8, c.shape), c)
    if layout == "token":
        byte = byte.swapaxes(1, 2)
    return torch.from_numpy(o4.pack(c)), torch.from_numpy(np.ascontiguousarray(byte))


class Batch4(Batch):
    """k, v, kp and vp are what the caches in 4 bits stand for; poisoned places have the scale 0xFF."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.k4, self.v4 = parts(self.kc, self.layout, 1), parts(self.vc, self.layout, 2)

        def held(x):
            return torch.from_numpy(o4.held(x)).to(self.dtype) if x.numel() else x

        self.k, self.v = [held(x) for x in self.k], [held(x) for x in self.v]
        self.kp, self.vp = held(self.kp), held(self.vp)
