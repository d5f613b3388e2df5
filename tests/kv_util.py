"""Batches for the tests of the paged cache operators: seeded inputs, a cache whose
pages lie in random order, and the float64 results with their error bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import kv as okv

BAD_PAGE = 1 << 30  # in places of the page table that no call may use


class Batch:
    """Sequences with q_lens new tokens and kv_lens keys; with `poison`, everything
    that no new token sees (page tails, unused pages, keys behind the window) is NaN
    and the table's unused entries name no page."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, head_dim, dtype, page_size=16, layout="token", window=0, sinks=0,
                 prefix=0, pad=0, seed=0, poison=True, scale=0.0, spread=1.0):
        assert len(q_lens) == len(kv_lens)
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(q_lens=q_lens, kv_lens=kv_lens, heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                             page_size=page_size, layout=layout, window=window, sinks=sinks, prefix=prefix, pad=pad,
                             poison=poison, scale=scale)
        self.group = heads // kv_heads
        self.real = sum(q_lens)
        self.tokens = self.real + pad
        cu = np.concatenate([[0], np.cumsum(q_lens)])
        self.cu_q = torch.tensor(cu, dtype=torch.int32)
        self.kv = torch.tensor(kv_lens, dtype=torch.int32)
        self.max_q = max(1, max(q_lens, default=1))

        def draw(n, mul=1.0):
            return (torch.randn(n, kv_heads, head_dim, generator=g) * mul).to(dtype)

        self.q = (torch.randn(self.tokens, heads, head_dim, generator=g) * spread).to(dtype)
        self.k = [draw(m) for m in kv_lens]
        self.v = [draw(m) for m in kv_lens]
        self.kp, self.vp = draw(prefix), draw(prefix)
        need = [-(-m // page_size) for m in kv_lens] + [-(-prefix // page_size)]
        self.num_pages = sum(need) + 3
        order = torch.randperm(self.num_pages, generator=g).tolist()
        cols = max([1] + need[:-1]) + 1
        self.table = torch.full((len(q_lens), cols), BAD_PAGE if poison else 0, dtype=torch.int32)
        shape = ((self.num_pages, page_size, kv_heads, head_dim) if layout == "token"
                 else (self.num_pages, kv_heads, page_size, head_dim))
        fill = math.nan if poison else 0.0
        self.kc, self.vc = torch.full(shape, fill, dtype=dtype), torch.full(shape, fill, dtype=dtype)
        for b, m in enumerate(kv_lens):
            first = m - q_lens[b]  # the first new token's position
            lo = max(0, first - window + 1) if window > 0 else 0
            seen = torch.zeros(m, dtype=torch.bool)
            if q_lens[b] > 0:
                seen[lo:] = True
                seen[:min(sinks, lo)] = True
            for c in range(need[b]):
                page = order.pop()
                a, e = c * page_size, min(c * page_size + page_size, m)
                if poison and not seen[a:e].any():
                    continue
                self.table[b, c] = page
                ok = seen[a:e] if poison else torch.ones(e - a, dtype=torch.bool)
                for cache, src in ((self.kc, self.k[b]), (self.vc, self.v[b])):
                    view = cache[page] if layout == "token" else cache[page].transpose(0, 1)
                    view[:e - a][ok] = src[a:e][ok]
        self.prefix_pages = torch.tensor([order.pop() for _ in range(need[-1])] + [BAD_PAGE], dtype=torch.int32)
        for c in range(need[-1]):
            a, e = c * page_size, min(c * page_size + page_size, prefix)
            for cache, src in ((self.kc, self.kp), (self.vc, self.vp)):
                view = cache[self.prefix_pages[c]] if layout == "token" else cache[self.prefix_pages[c]].transpose(0, 1)
                view[:e - a] = src[a:e]

    def keys(self, b, h):
        """Keys and values of sequence b, key head h, the prefix first."""
        return (np.concatenate([okv.to64(self.kp[:, h]), okv.to64(self.k[b][:, h])]),
                np.concatenate([okv.to64(self.vp[:, h]), okv.to64(self.v[b][:, h])]))

    def desc(self, cs, **kw):
        return cs.cs_kv_desc_init(**{**dict(
            dtype=self.dtype, heads=self.heads, kv_heads=self.kv_heads, head_dim=self.head_dim, page_size=self.page_size,
            num_pages=self.num_pages, cache_layout=self.layout, max_tokens=max(1, self.tokens), max_seqs=max(1, len(self.q_lens)),
            window=self.window, sinks=self.sinks, shared=1 if self.prefix else 0, scale=self.scale), **kw})

    def reference(self, tokens=None):
        """(out, lse, bound): float64, rows of `tokens` (default all real ones).

        bound, with u = eps / 2 of the dtype: the output's rounding u |O|; the
        weights' rounding, u sum(w |v|); their errors from the scores, sums of
        head_dim products in 32 bits (below 2^-12 absolute here, so 2^-11 relative
        with the sum's) and the accumulation of n products in 32 bits, n 2^-24
        sum(w |v|); and weights below the dtype's smallest steps, at most 2^-25
        of the row's largest weight for each of the n keys (fp16)."""
        u = torch.finfo(self.dtype).eps / 2
        scale = self.scale or 1.0 / math.sqrt(self.head_dim)
        rows = range(self.real) if tokens is None else tokens
        out = np.zeros((len(rows), self.heads, self.head_dim))
        lse = np.zeros((len(rows), self.heads))
        bound = np.zeros_like(out)
        cu = self.cu_q.tolist()
        q64 = okv.to64(self.q)
        cache = {}
        for i, t in enumerate(rows):
            b = max(x for x in range(len(self.q_lens)) if cu[x] <= t < cu[x + 1])
            pos = self.kv_lens[b] - self.q_lens[b] + t - cu[b]
            seen = okv.visible(pos, self.kv_lens[b], self.window, self.sinks, self.prefix)
            for h in range(self.heads):
                kh = h // self.group
                if (b, kh) not in cache:
                    cache[b, kh] = self.keys(b, kh)
                k, v = cache[b, kh]
                o, z, a = okv.attend(q64[t, h], k, v, seen, scale)
                n = int(seen.sum())
                out[i, h], lse[i, h] = o, z
                vmax = np.abs(v[seen]).max() if n else 0.0
                bound[i, h] = u * np.abs(o) + (u + 2.0 ** -11 + n * 2.0 ** -24) * a + n * 2.0 ** -25 * vmax + 1e-30
        return out, lse, bound


def rope_table(rows, rotary_dim, base=10000.0):
    r2 = rotary_dim // 2
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * base ** (-torch.arange(r2, dtype=torch.float64) / max(r2, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
