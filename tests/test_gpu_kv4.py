"""The paged cache in 4 bits on the GPU against the float64 definitions."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import consumer_gemm_chain_gb300 as cs
import oracle
from kv4_util import Batch4
from kv_util import BAD_PAGE, Batch, rope_table
from oracle import kv as okv
from oracle import kv4 as o4

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def cuda(pair):
    return tuple(x.cuda() for x in pair)


class Device:
    """A test batch on the GPU, with its plan."""

    def __init__(self, b: Batch4, **desc):
        self.b = b
        self.plan = cs.cs_kv_plan(b.desc(cs, **desc))
        self.cu_q, self.kv, self.table = b.cu_q.cuda(), b.kv.cuda(), b.table.cuda()
        self.q, self.k, self.v, self.prefix_pages = b.q.cuda(), cuda(b.k4), cuda(b.v4), b.prefix_pages.cuda()
        self.batch = cs.cs_kv_batch(self.plan, self.cu_q, self.kv, self.table, tokens=b.tokens, max_q=b.max_q)
        self.out = torch.full((b.tokens, b.heads, b.head_dim), 7.0, dtype=b.dtype, device="cuda")
        self.lse = torch.full((b.tokens, b.heads), 7.0, device="cuda")

    def attend(self, q=None, out=None, lse=True, stream=None):
        q, out = self.q if q is None else q, self.out if out is None else out
        lse = self.lse if lse else None
        if self.b.prefix:
            cs.cs_kv4_attention_shared(self.plan, self.batch, q, self.k, self.v, self.prefix_pages, self.b.prefix, out, lse,
                                       stream=stream)
        else:
            cs.cs_kv4_attention(self.plan, self.batch, q, self.k, self.v, out, lse, stream=stream)

    def ok(self):
        torch.cuda.synchronize()
        st = cs.cs_kv_status(self.plan)
        assert st == cs.CS_OK, f"{cs.STATUS_NAMES.get(st)}: {cs.cs_last_error_string()}"

    def check(self, tokens=None, out=None):
        """The outputs against the reference (rows `tokens`, default all), the padding untouched.  The bounds are those of
        the 16-bit cache: what 4 bits stand for are numbers of the dtype."""
        b = self.b
        ref, lse, bound = b.reference(tokens)
        rows = list(range(b.real)) if tokens is None else tokens
        full = (self.out if out is None else out).reshape(b.tokens, b.heads, b.head_dim)
        got = okv.to64(full)[rows]
        assert np.isfinite(got).all()
        err = np.abs(got - ref) / bound
        assert err.max(initial=0) <= 1, f"{err.max():.2f} of the bound at {np.unravel_index(err.argmax(), err.shape)}"
        got_lse = okv.to64(self.lse)[rows]
        empty = np.isneginf(lse)
        assert (np.isneginf(got_lse) == empty).all()
        # scores within 2^-12, the sum of n weights within n 2^-24, log in 32 bits
        assert np.abs(got_lse[~empty] - lse[~empty]).max(initial=0) <= 2.0 ** -11 + 2.0 ** -20 * np.abs(lse[~empty]).max(initial=0)
        assert (full[b.real:] == 7).all() and (self.lse[b.real:] == 7).all()


def run(b, **desc):
    d = Device(b, **desc)
    d.attend()
    d.ok()
    d.check()
    return d


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("heads,kv_heads,head_dim", [
    (128, 1, 64), (100, 1, 128), (12, 12, 128), (8, 2, 64), (28, 4, 128), (16, 1, 64), (6, 2, 128), (40, 2, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q,kv", [
    ([1], [1]), ([1], [2000]), ([1, 1, 0, 1], [17, 128, 5, 129]), ([4, 0, 1], [4, 0, 300]), ([2, 1], [70, 33]), ([5, 3], [700, 3]),
    ([130, 1, 33], [130, 257, 64]), ([257], [400])])
def test_attention(heads, kv_heads, head_dim, dtype, q, kv):
    run(Batch4(q, kv, heads, kv_heads, head_dim, dtype, pad=2, seed=len(q) + heads))


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("q,kv", [([1, 1], [333, 15]), ([3, 1], [99, 141]), ([150, 7], [333, 200])])
def test_pages_and_layouts(page_size, layout, q, kv):
    for heads, head_dim, dtype in ((8, 128, BF16), (8, 64, F16)):
        run(Batch4(q, kv, heads, 2, head_dim, dtype, page_size=page_size, layout=layout, seed=page_size))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 128), (129, 130), (1000, 5), (37, 1000)])
@pytest.mark.parametrize("q,kv", [([1, 1, 1], [900, 37, 140]), ([4, 2], [500, 41]), ([3, 300, 64], [500, 400, 901])])
def test_window_and_sinks(window, sinks, q, kv):
    run(Batch4(q, kv, 8, 2, 128, BF16, window=window, sinks=sinks, seed=window))
    run(Batch4(q, kv, 6, 6, 64, F16, window=window, sinks=sinks, seed=window, page_size=128, layout="head"))


@pytest.mark.parametrize("heads,kv_heads,head_dim,q,kv,window,sinks", [
    (12, 12, 128, [2226, 1517], [2226, 1517], 1024, 4), (8, 2, 64, [1900, 700, 1], [2500, 700, 3000], 700, 130),
    (12, 4, 128, [3000], [3000], 0, 0), (16, 1, 128, [640], [5000], 2000, 1)])
def test_many_items(heads, kv_heads, head_dim, q, kv, window, sinks):
    """More items than SMs, cut at places that depend on windows and sinks: rows at the
    borders of tiles and items, and some between."""
    d = Device(Batch4(q, kv, heads, kv_heads, head_dim, F16, window=window, sinks=sinks, seed=window))
    d.attend()
    d.ok()
    rows, at = [], 0
    for n in q:
        rows += [at + i for i in range(n) if i % 128 in (0, 127) or i % 85 == 84]
        at += n
    d.check(rows)


@pytest.mark.parametrize("heads,kv_heads,head_dim,q,kv,window,sinks", [
    (8, 2, 128, [600, 1, 70], [6000, 3900, 4100], 0, 0), (8, 8, 64, [600, 70, 0, 1], [6000, 4100, 0, 3900], 3400, 130),
    (16, 1, 128, [40, 300], [9000, 4000], 3300, 4)])
@pytest.mark.parametrize("num_sms", [0, 37])
def test_long_items(heads, kv_heads, head_dim, q, kv, window, sinks, num_sms):
    """Items long enough to be cut and joined, and shorter ones between them."""
    d = Device(Batch4(q, kv, heads, kv_heads, head_dim, BF16, window=window, sinks=sinks, seed=kv[0], page_size=64), num_sms=num_sms)
    d.attend()
    d.ok()
    rows, at = [], 0
    for n in q:
        rows += [at + i for i in range(n) if i % 64 in (0, 63) or i == n - 1]
        at += n
    d.check(rows)


@pytest.mark.parametrize("lens", [[512] * 6, [1024, 90, 700, 2, 511], [256], [20] * 90])
def test_whole_items(lens):
    """Prompts short enough for no item to be cut: about as many items as SMs, fewer and more."""
    d = Device(Batch4(lens, lens, 12, 12, 128, F16, seed=len(lens)))
    for _ in range(2):
        d.out.fill_(7), d.lse.fill_(7)
        d.attend()
    d.ok()
    rows, at = [], 0
    for n in lens:
        rows += [at + i for i in range(n) if i % 128 in (0, 127) or i == n - 1]
        at += n
    d.check(rows)


@pytest.mark.parametrize("heads,kv_heads,num_sms", [(14, 7, 0), (14, 7, 15), (64, 64, 20), (64, 32, 0), (9, 3, 6)])
@pytest.mark.parametrize("q,kv", [([1] * 3, [700, 5, 1300]), ([1] * 35, [9 * i + 1 for i in range(35)]), ([2, 0, 1], [400, 9, 90])])
def test_division_by_heads(heads, kv_heads, num_sms, q, kv):
    """Key heads that share the CTAs out evenly, with some left over, and more heads than CTAs."""
    for head_dim, dtype in ((64, BF16), (128, F16)):
        run(Batch4(q, kv, heads, kv_heads, head_dim, dtype, seed=heads), num_sms=num_sms)


@pytest.mark.parametrize("prefix", [1, 16, 127, 500, 2049])
@pytest.mark.parametrize("q,kv", [([1] * 5, [1, 40, 130, 2, 16]), ([1, 0, 3], [9, 0, 3]), ([40, 1, 70], [40, 300, 75]), ([2], [1])])
def test_shared_prefix(prefix, q, kv):
    run(Batch4(q, kv, 8, 2, 128, BF16, prefix=prefix, pad=3, seed=prefix))
    run(Batch4(q, kv, 7, 1, 64, F16, prefix=prefix, page_size=64, layout="head", seed=prefix))


def test_a_prefix_of_no_keys():
    b = Batch4([1, 30], [50, 70], 8, 2, 128, BF16)
    d = Device(b, shared=1)
    cs.cs_kv4_attention_shared(d.plan, d.batch, d.q, d.k, d.v, d.prefix_pages, 0, d.out, d.lse)
    d.ok()
    d.check()


def test_tokens_before_position_zero():
    for q, kv in (([4, 3], [2, 0]), ([200, 1], [60, 0])):
        d = run(Batch4(q, kv, 8, 2, 128, BF16))
        assert (d.out[:q[0] - kv[0]] == 0).all()
        run(Batch4(q, kv, 4, 4, 64, F16, window=8, sinks=2))


@pytest.mark.parametrize("q,kv,rows", [([1, 1], [40000, 9000], None), ([700, 1], [9001, 5000], [0, 1, 350, 699, 700]),
                                       ([3], [30001], None)])
def test_long_contexts(q, kv, rows):
    d = Device(Batch4(q, kv, 8, 2, 128, BF16, page_size=64, seed=3))
    d.attend()
    d.ok()
    d.check(rows)


def test_many_sequences():
    run(Batch4([1] * 3001, [5] * 3000 + [40], 2, 1, 64, F16))
    run(Batch4([0, 1] * 900, [3, 4] * 900, 2, 2, 64, BF16, poison=False))
    r = np.random.default_rng(0)
    run(Batch4([1] * 700, [int(x) for x in r.integers(1, 90, 700)], 4, 2, 64, F16))
    q = [int(x) for x in r.integers(0, 9, 300)]
    run(Batch4(q, [n + int(x) for n, x in zip(q, r.integers(0, 60, 300))], 4, 2, 64, BF16))


@pytest.mark.parametrize("dtype,size", [(F16, 9000.0), (F16, 1e-4), (BF16, 3e4), (BF16, 1e-4)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_values_of_other_sizes(dtype, size, n):
    """Scales near the ends of their range: values of up to four and a half times `size`, in f16 up to 4e4."""
    b = Batch4([n], [300], 8, 2, 64, dtype, seed=n)
    v = (b.vc.float() * size).to(dtype)
    from kv4_util import parts
    b.v4 = parts(v, b.layout)
    g = o4.held(v)
    b.v = [torch.stack([torch.from_numpy(g[int(b.table[0, j // 16]), j % 16]) for j in range(300)]).to(dtype)]
    d = Device(b)
    d.attend()
    d.ok()
    d.check()


def scaled_batch(q, kv, dtype, sizes_k, sizes_v, head_dim=64, **kw):
    """A batch whose keys' and values' groups are of the sizes given, in turn."""
    from kv4_util import parts
    b = Batch4(q, kv, 8, 2, head_dim, dtype, **kw)

    def scaled(cache, sizes):
        groups = cache.float().unflatten(-1, (-1, 32))
        s = torch.tensor(sizes)[torch.arange(groups[..., 0].numel()) % len(sizes)].view(groups.shape[:-1])
        x = (groups * s[..., None]).flatten(-2)
        return x.clamp(-6e4, 6e4).to(dtype) if dtype == F16 else x.to(dtype)  # (f16 ends at 65504)

    for name, cache, sizes, seqs in (("k4", b.kc, sizes_k, b.k), ("v4", b.vc, sizes_v, b.v)):
        x = scaled(cache, sizes)
        setattr(b, name, parts(x, b.layout))
        held = torch.from_numpy(o4.held(x)).to(dtype)
        for i, m in enumerate(kv):
            for j in range(m):
                if int(b.table[i, j // 16]) != BAD_PAGE:
                    seqs[i][j] = held[int(b.table[i, j // 16]), j % 16]
    return b


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("dtype,big", [(F16, 1.4e4), (BF16, 9e4), (BF16, 1.3e4)])
def test_scales_of_all_sizes_beside_one_another(n, dtype, big):
    """Groups of values near the ends of the scales' range, of usual ones and of zeros, in one key and in neighbouring ones."""
    sizes = [big, 1.0, 1e-5, 300.0, 0.0, 1e-4, big, 3e-6, 0.03, 1e3, 20.0]
    run(scaled_batch([n, 1], [200, 90], dtype, [1.0], sizes, seed=n))
    run(scaled_batch([n, 1], [200, 90], dtype, [1.0, 0.3], sizes, head_dim=128, seed=n))
    # keys of such sizes: scores of a few units by the scale, weights over the keys with large groups only
    b = scaled_batch([n], [150], dtype, sizes, [1.0], seed=n, scale=2.0 ** -19, spread=1.0)
    d = Device(b)
    d.attend()
    d.ok()
    ref, lse, bound = b.reference()
    # 64 products in 32 bits: a score is off by up to 2^-24 * 64 * sum |q k| scale
    worst = 2 * 2.0 ** -24 * 64 * 64 * float(b.q.float().abs().amax() * b.k[0].float().abs().amax()) * 2.0 ** -19
    assert (np.abs(okv.to64(d.out) - ref) <= bound * (1 + worst / 2.0 ** -11)).all()


def test_large_scores():
    """Rows whose maximum keeps rising by much, and weights far below the row's largest."""
    for n in (1, 2, 200):
        for dtype in (BF16, F16):
            b = scaled_batch([n], [600], dtype, [float(x) for x in np.linspace(0.02, 3, 61)], [1.0], head_dim=128, scale=1.0, seed=5)
            d = Device(b)
            d.attend()
            d.ok()
            ref, _, bound = b.reference()
            worst = 2 * 2.0 ** -24 * 128 * 128 * float(b.q.float().abs().amax() * b.k[0].float().abs().amax())
            assert (np.abs(okv.to64(d.out) - ref) <= bound * (1 + worst / 2.0 ** -11)).all()


@pytest.mark.parametrize("size", [1e-30, 1e-6, 3e4, 1e30])
@pytest.mark.parametrize("n", [1, 4])
def test_queries_of_other_sizes(n, size):
    """Rows of bf16 queries far from 1, the scale undoing it; rows of one call differ, and values within a row too."""
    b = Batch4([n, 1], [300, 80], 8, 2, 128, BF16, seed=n, scale=float(np.float32(0.09 / size)))
    b.q = (b.q.float() * size).to(BF16)
    b.q[..., 1::7] *= 2.0 ** -20
    b.q[0, 1::2] *= 2.0 ** -12
    run(b)


def test_a_query_that_is_not_finite():
    """Its rows are NaN; the others of the call are as without it."""
    for n in (1, 2, 30):
        for dtype in (F16, BF16):
            b = Batch4([n, n], [200, 100], 8, 2, 128, dtype, seed=n)
            d = Device(b)
            d.attend()
            d.ok()
            clean = d.out.clone()
            d.q[0, 1, 5], d.q[n, 6, 7] = math.nan, math.inf
            d.attend()
            d.ok()
            assert torch.isnan(d.out[0, 1]).all() and torch.isnan(d.out[n, 6]).all()
            d.out[0, 1], d.out[n, 6] = clean[0, 1], clean[n, 6]
            assert torch.equal(d.out, clean)


@pytest.mark.parametrize("q,kv", [([4, 1], [70, 9]), ([3], [900]), ([200, 30], [300, 30]), ([130], [2000]), ([2], [40])])
@pytest.mark.parametrize("window,prefix", [(0, 0), (33, 0), (0, 50)])
def test_scales_that_are_no_number_at_keys_hidden_from_some_rows(q, kv, window, prefix):
    """Values of a group at keys that only later tokens (or, under a window, only earlier ones) see: every other
    row is as if they were not there; rows that see one are NaN in the group's dimensions and right elsewhere."""
    for dtype in (BF16, F16):
        b = Batch4(q, kv, 8, 2, 128, dtype, window=window, sinks=2 if window else 0, prefix=prefix, seed=kv[0])
        spoilt = []  # (sequence, key): seen by the last token only, and by the first only
        for s, (n, m) in enumerate(zip(q, kv)):
            spoilt.append((s, m - 1))
            if window and m - n - window + 1 >= 2 and n > 1:
                spoilt.append((s, m - n - window + 1))
        for s, j in spoilt:
            b.v4[1][int(b.table[s, j // 16]), :, j % 16, 2] = 0xFF
            b.v[s][j, :, 64:96] = 0.0  # rows that do not see it never read it
        d = Device(b)
        for _ in range(2):  # the marks of the first call are cleared
            d.out.fill_(7), d.lse.fill_(7)
            d.attend()
        d.ok()
        ref, lse, bound = b.reference()
        got, t = okv.to64(d.out), 0
        assert np.abs(okv.to64(d.lse) - lse).max() <= 2.0 ** -11 + 2.0 ** -20 * np.abs(lse).max()
        for s, (n, m) in enumerate(zip(q, kv)):
            for i in range(n):
                p = m - n + i
                hit = any(x == s and j <= p and (not window or j > p - window) for x, j in spoilt)
                ok = np.ones(128, dtype=bool)
                ok[64:96] = not hit
                assert (np.abs(got[t, :, ok] - ref[t, :, ok]) <= bound[t, :, ok]).all(), (s, i)
                assert not hit or np.isnan(got[t, :, 64:96]).all(), (s, i)
                t += 1


@pytest.mark.parametrize("q,kv", [([4], [70]), ([200], [300])])
def test_keys_that_are_no_number_where_hidden(q, kv):
    b = Batch4(q, kv, 8, 2, 64, BF16)
    n, m = q[0], kv[0]
    b.k4[1][int(b.table[0, (m - 1) // 16]), :, (m - 1) % 16, 1] = 0xFF
    d = Device(b)
    d.attend()
    d.ok()
    ref, _, bound = b.reference(list(range(n - 1)))
    got = okv.to64(d.out)
    assert (np.abs(got[:n - 1] - ref) <= bound).all() and np.isnan(got[n - 1]).all()


def test_rows_of_other_strides():
    b = Batch4([1, 90, 3], [50, 90, 700], 8, 2, 128, BF16, pad=2)
    d = Device(b)
    wide = torch.full((b.tokens, 8 * 128 + 40), 7.0, dtype=BF16, device="cuda")
    q = torch.zeros(b.tokens, 8 * 128 + 24, dtype=BF16, device="cuda")
    q[:, 8:8 + 1024] = d.q.flatten(1)
    out = wide[:, 32:32 + 1024]
    d.attend(q[:, 8:8 + 1024], out)
    d.ok()
    d.check(out=out)
    assert (wide[:, :32] == 7).all() and (wide[:, 1056:] == 7).all()


def test_same_bits_on_every_call():
    for b in (Batch4([1] * 9, [900, 5, 77, 3000, 1, 128, 129, 2000, 64], 16, 2, 128, BF16),
              Batch4([300, 1, 50], [900, 3000, 50], 8, 2, 64, F16),
              Batch4([1] * 20, list(range(1, 21)), 8, 2, 128, BF16, prefix=1000)):
        d = Device(b)
        d.attend()
        first, lse = d.out.clone(), d.lse.clone()
        for _ in range(5):
            d.out.zero_()
            d.attend()
            assert torch.equal(first[:b.real], d.out[:b.real]) and torch.equal(lse, d.lse)
        d.ok()


def test_fewer_sms_and_no_lse():
    for sms in (1, 7):
        d = Device(Batch4([1, 60], [300, 700], 8, 2, 128, BF16), num_sms=sms)
        d.attend()
        d.ok()
        d.check()
        d.out.fill_(7)
        d.attend(lse=False)
        d.ok()
        d.check()
        d = Device(Batch4([1, 2], [300, 700], 8, 2, 64, F16), num_sms=sms)
        d.attend()
        d.ok()
        d.check()


# ------------------------------------------------------------------ append and read
def rotated(x, rope, angles, heads, hk, d, rotary, pairing):
    """Rows [tokens, heads + 2 hk, d] with Q and K rotated in 32 bits, each operation rounded, then to the dtype."""
    y = x.float().numpy().reshape(-1, heads + 2 * hk, d).copy()
    if rotary:
        t = rope.numpy()[angles][:, None]
        cos, sin = t[..., :rotary // 2], t[..., rotary // 2:]
        i = np.arange(rotary // 2)
        lo, hi = (i, i + rotary // 2) if pairing == "half" else (2 * i, 2 * i + 1)
        a, b = y[:, :heads + hk][..., lo].copy(), y[:, :heads + hk][..., hi].copy()
        y[:, :heads + hk, lo] = a * cos - b * sin
        y[:, :heads + hk, hi] = b * cos + a * sin
    return torch.from_numpy(y).to(x.dtype)


def append_case(q, kv, heads, hk, d, dtype, rotary, pairing, layout, page_size, pad=0, in_place=False, positions=False, shift=0,
                spoil=False):
    b = Batch4(q, kv, heads, hk, d, dtype, page_size=page_size, layout=layout, pad=pad, seed=rotary + d)
    dev = Device(b, rotary_dim=rotary, rotary_pairing=pairing)
    g = torch.Generator().manual_seed(9)
    width = (heads + 2 * hk) * d
    sizes = torch.exp2(torch.randint(-30, 14 if dtype == F16 else 40, (b.tokens, width // 32, 1), generator=g).float())
    store = torch.randn(b.tokens, width + shift, generator=g)
    store[:, :width] *= torch.where(torch.rand(b.tokens, width // 32, 1, generator=g) < 0.2, sizes, 1.0).expand(-1, -1, 32).flatten(1)
    store = store.clamp(-6e4, 6e4).to(dtype) if dtype == F16 else store.to(dtype)
    if spoil:
        store[0, heads * d + 3], store[-1 - pad, width - 5], store[0, width - 40] = math.nan, math.inf, -math.inf
        store[1, heads * d:width] = 0
    qkv = store[:, :width]
    rows = max(kv) + 50
    rope = rope_table(rows, rotary) if rotary else None
    pos_of, where = [], []
    for s, (n, m) in enumerate(zip(q, kv)):
        pos_of += list(range(m - n, m))
        where += [(s, p) for p in range(m - n, m)]
    ids = torch.randint(0, rows, (b.tokens,), generator=g, dtype=torch.int32) if positions else None
    before = [x.clone() for x in (*dev.k, *dev.v)]
    dstore = store.cuda()
    dqkv = dstore[:, :width]
    q_out = dqkv[:, :heads * d] if in_place else torch.full((b.tokens, heads, d), 7.0, dtype=dtype, device="cuda")
    cs.cs_kv4_append(dev.plan, dev.batch, dqkv, q_out, dev.k, dev.v, rope=None if rope is None else rope.cuda(),
                     positions=None if ids is None else ids.cuda())
    dev.ok()
    angles = ids.numpy() if positions else np.maximum(np.array(pos_of + [0] * pad), 0)
    want = rotated(qkv, rope, angles, heads, hk, d, rotary, pairing)
    live = [i for i, p in enumerate(pos_of) if p >= 0]
    same = lambda a, c: torch.equal(a.contiguous().view(torch.int16), c.contiguous().view(torch.int16))  # noqa: E731
    got_q = q_out.reshape(b.tokens, heads, d).cpu()
    finite = torch.isfinite(want[:, :heads])
    assert torch.equal(got_q[live][finite[live]], want[live, :heads][finite[live]])
    if in_place:
        assert same(dstore[:, heads * d:].cpu(), store[:, heads * d:]) and same(dstore[b.real:].cpu(), store[b.real:])
    else:
        assert (q_out[b.real:] == 7).all()
    # the bytes at the tokens' places, and nothing else changed
    for cache, first, mine in ((dev.k, heads, before[:2]), (dev.v, heads + hk, before[2:])):
        codes, scales = (x.cpu() for x in mine)
        c, byte = o4.quantise(want[:, first:first + hk])
        packed, byte = torch.from_numpy(o4.pack(c)), torch.from_numpy(byte)
        for i in live:
            s, p = where[i]
            page, slot = int(b.table[s, p // page_size]), p % page_size
            codes[(page, slot) if layout == "token" else (page, slice(None), slot)] = packed[i]
            scales[page, :, slot] = byte[i]
        assert torch.equal(cache[1].cpu(), scales)
        assert torch.equal(cache[0].cpu(), codes)
    # and read back
    k_out, v_out = (torch.full((b.tokens, hk, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    cs.cs_kv4_read(dev.plan, dev.batch, dev.k, dev.v, k_out, v_out)
    dev.ok()
    for out, first in ((k_out, heads), (v_out, heads + hk)):
        ref = np.full((b.tokens, hk, d), 7.0)
        ref[live] = o4.held(want[:, first:first + hk])[live]
        np.testing.assert_array_equal(okv.to64(out), ref)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,hk,d,rotary,pairing", [
    (12, 12, 128, 128, "half"), (8, 2, 64, 64, "adjacent"), (28, 4, 128, 32, "half"), (6, 1, 64, 16, "adjacent"),
    (5, 5, 128, 112, "half"), (3, 3, 64, 48, "half"), (4, 2, 64, 0, "half")])
@pytest.mark.parametrize("q,kv", [([1], [1]), ([1, 0, 1, 1], [16, 40, 17, 300]), ([130, 3, 40], [140, 3, 95])])
def test_append(dtype, heads, hk, d, rotary, pairing, q, kv):
    append_case(q, kv, heads, hk, d, dtype, rotary, pairing, "token", 16, pad=3)


@pytest.mark.parametrize("layout,page_size", [("head", 16), ("token", 128), ("head", 64)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("positions", [False, True])
def test_append_forms(layout, page_size, in_place, positions):
    for pairing in ("half", "adjacent"):
        append_case([1, 70, 0, 5], [9, 200, 3, 5], 8, 2, 128, BF16, 64, pairing, layout, page_size, pad=2, in_place=in_place,
                    positions=positions, shift=24)
    append_case([1], [9], 8, 2, 128, BF16, 64, "half", layout, page_size, in_place=in_place, positions=positions)


def test_append_of_values_that_are_not_finite_and_of_zeros():
    append_case([30, 5], [40, 5], 8, 2, 128, BF16, 0, "half", "head", 32, pad=1, spoil=True)
    append_case([30, 5], [40, 5], 8, 2, 64, F16, 0, "half", "token", 16, spoil=True)


def test_append_leaves_out_tokens_before_position_zero():
    append_case([5, 2], [3, 0], 8, 2, 64, F16, 64, "half", "token", 16)


def test_append_of_ties():
    """Magnitudes at the middle between two scales, and values at the middle between two codes, in every binade of f16."""
    rows = []
    for byte in range(1, 0xF4):
        s, up = o4.SCALES[byte], o4.SCALES[byte + 1]
        mid = 7 * (s + up) / 2
        x = np.zeros(64)
        x[:16] = np.arange(-8, 8) * s + s / 2
        x[7], x[15] = 0, 7 * s
        x[:16] = np.clip(x[:16], -7 * s, 7 * s)
        x[32] = mid
        rows.append(x)
    x = np.stack(rows)
    for dtype in (F16, BF16):
        t = torch.from_numpy(x).to(dtype)
        keep = (okv.to64(t) == x).all(1) & np.isfinite(okv.to64(t)).all(1)
        assert keep.sum() > 100
        t = t[torch.from_numpy(keep)]
        n = len(t)
        b = Batch4([n], [n], 1, 1, 64, dtype)
        d = Device(b)
        qkv = t.repeat(1, 3).cuda()
        out = torch.empty(n, 64, dtype=dtype, device="cuda")
        cs.cs_kv4_append(d.plan, d.batch, qkv, out, d.k, d.v)
        k, v = (torch.empty(n, 1, 64, dtype=dtype, device="cuda") for _ in range(2))
        cs.cs_kv4_read(d.plan, d.batch, d.k, d.v, k, v)
        d.ok()
        np.testing.assert_array_equal(okv.to64(k)[:, 0], o4.held(t))
        assert torch.equal(k, v)


@pytest.mark.parametrize("dtype,d", [(F16, 64), (BF16, 128)])
def test_read_of_every_byte(dtype, d):
    """All scales and codes, those that no append writes among them."""
    b = Batch4([256], [256], 2, 1, d, dtype, poison=False)
    dev = Device(b)
    g = np.random.default_rng(1)
    c = g.integers(-8, 8, (b.num_pages, 16, 1, d)).astype(np.int8)
    byte = g.permutation(np.arange(b.num_pages * 16) % 256).reshape(b.num_pages, 1, 16, 1).repeat(d // 32, -1).astype(np.uint8)
    cache = torch.from_numpy(o4.pack(c)).cuda(), torch.from_numpy(np.ascontiguousarray(byte)).cuda()
    k = torch.empty(256, 1, d, dtype=dtype, device="cuda")
    cs.cs_kv4_read(dev.plan, dev.batch, cache, cache, k, None)
    dev.ok()
    with np.errstate(invalid="ignore"):
        values = o4.values(c, byte.swapaxes(1, 2))
    want = np.stack([values[int(b.table[0, j // 16]), j % 16] for j in range(256)])
    got = okv.to64(k)
    named = np.isfinite(want)
    fits = np.abs(np.where(named, want, 0)) <= torch.finfo(dtype).max
    assert (got[named & fits] == want[named & fits]).all()
    assert not np.isfinite(got[~named]).all()


def test_read_of_whole_sequences_and_of_parts():
    heads, hk, d = 4, 2, 128
    for layout, page_size in (("token", 16), ("head", 64)):
        kv = [300, 1, 0, 77, 16]
        b = Batch4(kv, kv, heads, hk, d, BF16, layout=layout, page_size=page_size, pad=3, poison=False)
        dev = Device(b)
        wide = torch.full((b.tokens, hk * d + 24), 7.0, dtype=BF16, device="cuda")
        v_out = torch.full((b.tokens, hk, d), 7.0, dtype=BF16, device="cuda")
        cs.cs_kv4_read(dev.plan, dev.batch, dev.k, dev.v, wide[:, 8:8 + hk * d], v_out)
        dev.ok()
        assert torch.equal(wide[:b.real, 8:8 + hk * d].cpu(), torch.cat(b.k).flatten(1))
        assert torch.equal(v_out[:b.real].cpu(), torch.cat(b.v))
        assert (wide[:, :8] == 7).all() and (wide[:, 8 + hk * d:] == 7).all() and (wide[b.real:] == 7).all() and (v_out[b.real:] == 7).all()
        # the last keys of some sequences, values only
        n = [5, 1, 0, 0, 16]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        part = cs.cs_kv_batch(dev.plan, cu, dev.kv, dev.table, tokens=22, max_q=16)
        out = torch.full((22, hk, d), 7.0, dtype=BF16, device="cuda")
        cs.cs_kv4_read(dev.plan, part, None, dev.v, None, out)
        dev.ok()
        assert torch.equal(out.cpu(), torch.cat([v[len(v) - i:] for i, v in zip(n, b.v)]))


# ------------------------------------------------------------------ together
def test_a_run_of_steps():
    """Prompts and then single tokens of three sequences: append, attention under a window, reading back; beside a
    16-bit cache that the same plan serves.  Against the definitions over everything appended."""
    heads, hk, d, window, sinks, dtype = 8, 2, 64, 50, 3, BF16
    r = np.random.default_rng(2)
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=hk, head_dim=d, page_size=16, num_pages=40,
                                            max_tokens=300, max_seqs=3, rotary_dim=32, window=window, sinks=sinks))
    codes, scales = cs.cs_kv4_shapes(plan)
    k, v = ((torch.full(codes, 0x5A, dtype=torch.uint8, device="cuda"), torch.full(scales, 0xFF, dtype=torch.uint8, device="cuda"))
            for _ in range(2))
    kc, vc = (torch.full(plan.cache_shape, math.nan, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.from_numpy(r.permutation(40)[:36].reshape(3, 12).astype(np.int32)).cuda()
    rope = rope_table(200, 32)
    lens, keys, vals = [0, 0, 0], [[], [], []], [[], [], []]
    u = torch.finfo(dtype).eps / 2
    for step in ([100, 1, 0], [1, 0, 130], [1, 1, 1], [20, 3, 1], [1, 1, 1]):
        lens = [m + n for m, n in zip(lens, step)]
        T = sum(step)
        qkv = torch.from_numpy(r.standard_normal((T, (heads + 2 * hk) * d))).to(dtype)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(step)]), dtype=torch.int32, device="cuda")
        batch = cs.cs_kv_batch(plan, cu, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, tokens=T, max_q=max(step))
        work, q16 = qkv.cuda(), torch.empty(T, heads, d, dtype=dtype, device="cuda")
        out, out16, k_out = (torch.empty(T, n, d, dtype=dtype, device="cuda") for n in (heads, heads, hk))
        cs.cs_kv_append(plan, batch, work, q16, kc, vc, rope=rope.cuda())
        cs.cs_kv4_append(plan, batch, work, work[:, :heads * d], k, v, rope=rope.cuda())
        cs.cs_kv4_attention(plan, batch, work[:, :heads * d], k, v, out)
        cs.cs_kv_attention(plan, batch, q16, kc, vc, out16)
        cs.cs_kv4_read(plan, batch, k, v, k_out, None)
        torch.cuda.synchronize()
        assert cs.cs_kv_status(plan) == cs.CS_OK
        angles = np.concatenate([np.arange(m - n, m) for n, m in zip(step, lens)])
        want = rotated(qkv, rope, angles, heads, hk, d, 32, "half")
        k_held, v_held = o4.held(want[:, heads:heads + hk]), o4.held(want[:, heads + hk:])
        np.testing.assert_array_equal(okv.to64(k_out), k_held)
        assert torch.isfinite(out16).all() and float((out16.float() - out.float()).abs().max()) < 2.5
        got, i = okv.to64(out), 0
        for s, n in enumerate(step):
            keys[s] += list(k_held[i:i + n])
            vals[s] += list(v_held[i:i + n])
            for p in range(lens[s] - n, lens[s]):
                seen = okv.visible(p, lens[s], window, sinks)
                for h in range(heads):
                    o, _, a = okv.attend(okv.to64(want[i, h]), np.array([y[h // 4] for y in keys[s]]),
                                         np.array([y[h // 4] for y in vals[s]]), seen, d ** -0.5)
                    # output and weights rounded, scores and sums in 32 bits
                    assert (np.abs(got[i, h] - o) <= u * np.abs(o) + (u + 2.0 ** -11 + len(seen) * 2.0 ** -24) * a + 1e-30).all()
                i += 1


def test_prompt_then_tokens_through_an_attention_chain():
    """A prompt and then single tokens through cs_attn_cached4_forward equal the stages called one by one, bit by bit, and
    the whole sequence's attention over held keys and values."""
    H, heads, dtype = 256, 2, F16
    F, total, prompt = heads * 128, 40, 33
    g = torch.Generator().manual_seed(4)
    X = (torch.randn(total, H, generator=g) * 0.5).to(dtype)
    Wqkv = (torch.randn(H, 3 * F, generator=g) * 0.06).to(dtype)
    Wo = (torch.randn(F, H, generator=g) * 0.06).to(dtype)
    rope = rope_table(total, 128).cuda()
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=heads, num_pages=4, max_tokens=prompt, max_seqs=1,
                                            rotary_dim=128))
    codes, scales = cs.cs_kv4_shapes(plan)
    k, v = ((torch.zeros(codes, dtype=torch.uint8, device="cuda"), torch.full(scales, 0xFF, dtype=torch.uint8, device="cuda"))
            for _ in range(2))
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    qkv = okv.to64(X) @ okv.to64(Wqkv)
    done = 0
    for n in [prompt] + [1] * (total - prompt):
        desc = cs.cs_chain_desc_init(kind="attn", M=n, H=H, F=F, dtype=dtype, heads=heads, head_dim=128, split_k=1, sk_tiles=-1)
        with cs.cs_chain_plan(desc) as chain:
            batch = cs.cs_kv_batch(plan, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                   torch.tensor([done + n], dtype=torch.int32, device="cuda"), table, tokens=n, max_q=n)
            Y = torch.empty(n, H, dtype=dtype, device="cuda")
            for _ in range(2):  # a step may be run again
                cs.cs_attn_cached4_forward(chain, plan, batch, X[done:done + n].cuda(), Wqkv.cuda(), Wo.cuda(), Y, k, v, rope=rope)
            torch.cuda.synchronize()
            assert cs.cs_chain_status(chain) == cs.CS_OK and cs.cs_kv_status(plan) == cs.CS_OK
        done += n
        # the keys and values that the cache holds now, and attention over them in 64 bits
        whole = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=heads, num_pages=4, max_tokens=total, max_seqs=1))
        rows = cs.cs_kv_batch(whole, torch.tensor([0, done], dtype=torch.int32, device="cuda"),
                              torch.tensor([done], dtype=torch.int32, device="cuda"), table, tokens=done, max_q=done)
        K, V = (torch.empty(done, heads, 128, dtype=dtype, device="cuda") for _ in range(2))
        cs.cs_kv4_read(whole, rows, k, v, K, V)
        torch.cuda.synchronize()
        K, V = okv.to64(K), okv.to64(V)
        t = okv.to64(rope.cpu())[:, None]
        q = okv.rotate(qkv.reshape(total, 3 * heads, 128)[:, :heads], t[..., :64], t[..., 64:], "half")
        O = np.zeros((n, heads, 128))
        for i in range(n):
            for h in range(heads):
                O[i, h] = okv.attend(q[done - n + i, h], K[:, h], V[:, h], okv.visible(done - n + i, done, 0, 0), 128 ** -0.5)[0]
        assert oracle.rel_err(Y.cpu(), O.reshape(n, F) @ okv.to64(Wo)) <= 5e-3
        # what is held is within a little more than half a step of the exact keys (and of their own rounding)
        exact = okv.rotate(qkv.reshape(total, 3 * heads, 128)[:done, heads:2 * heads], t[:done, :, :64], t[:done, :, 64:], "half")
        step = np.abs(exact).reshape(done, heads, 4, 32).max(-1).repeat(32, -1) / 7
        assert (np.abs(K - exact) <= 0.6 * step + 1e-3).all()


def test_a_captured_step_with_other_lengths():
    """Append, attention and reading captured once, replayed as a sequence grows, on the stream of the replay."""
    heads, hk, d = 8, 2, 128
    for n in (1, 3, 20):
        full = Batch4([n, n], [300 + n, 70 + n], heads, hk, d, BF16, poison=False, seed=n)
        dev = Device(full, rotary_dim=0)
        qkv = torch.cat([full.q.flatten(1), torch.cat([k[-n:].flatten(1) for k in full.k]),
                         torch.cat([v[-n:].flatten(1) for v in full.v])], 1).cuda()
        q_out = torch.zeros_like(dev.q)
        k_out, v_out = (torch.zeros(2 * n, hk, d, dtype=BF16, device="cuda") for _ in range(2))

        def step():
            cs.cs_kv4_append(dev.plan, dev.batch, qkv, q_out, dev.k, dev.v)
            cs.cs_kv4_attention(dev.plan, dev.batch, q_out, dev.k, dev.v, dev.out, dev.lse)
            cs.cs_kv4_read(dev.plan, dev.batch, dev.k, dev.v, k_out, v_out)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        dev.ok()
        want = [x.clone() for x in (dev.out, dev.lse, k_out, v_out)]
        saved = [x.clone() for x in (*dev.k, *dev.v)]
        dev.kv.copy_(torch.tensor([40, 20 + n], dtype=torch.int32))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graph.replay()
        dev.ok()
        dev.kv.copy_(full.kv)
        for x, y in zip((*dev.k, *dev.v), saved):
            x.copy_(y)
        for x in (dev.out, dev.lse, k_out, v_out):
            x.fill_(7)
        with torch.cuda.stream(side):
            graph.replay()
        dev.ok()
        for x, y in zip((dev.out, dev.lse, k_out, v_out), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("q,kv,prefix", [([1] * 40, [1 + 9 * i for i in range(40)], 3001), ([1, 3, 2], [400, 90, 2], 700),
                                         ([1], [200], 40), ([90, 1], [300, 20], 1000)])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_right_behind_one_another(q, kv, prefix, captured):
    """Kernels start while the ones before them end: the same results, bit by bit, as with nothing else running
    (append, attention behind a prefix, attention, reading; again with other tokens)."""
    b = Batch4(q, kv, 8, 2, 128, BF16, prefix=prefix, seed=prefix)
    d = Device(b, rotary_dim=0)
    g = torch.Generator().manual_seed(5)
    n = 6
    qkv = torch.randn(n, b.tokens, 12 * 128, generator=g).to(BF16).cuda()
    outs = torch.zeros(2, n, 2, b.tokens, 8, 128, dtype=BF16, device="cuda")
    read = torch.zeros(2, n, 2, b.tokens, 2, 128, dtype=BF16, device="cuda")
    qs = torch.zeros(2, b.tokens, 8, 128, dtype=BF16, device="cuda")

    def step(i, out, back, pause):
        cs.cs_kv4_append(d.plan, d.batch, qkv[i], qs[i % 2], d.k, d.v)
        pause()
        cs.cs_kv4_attention_shared(d.plan, d.batch, qs[i % 2], d.k, d.v, d.prefix_pages, b.prefix, out[0])
        pause()
        cs.cs_kv4_attention(d.plan, d.batch, qs[i % 2], d.k, d.v, out[1])
        pause()
        cs.cs_kv4_read(d.plan, d.batch, d.k, d.v, back[0], back[1])
        pause()

    for i in range(n):
        step(i, outs[0, i], read[0, i], torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            for i in range(n):
                step(i, outs[1, i], read[1, i], lambda: None)
    for _ in range(3):
        outs[1].fill_(7), read[1].fill_(7)
        if captured:
            graph.replay()
        else:
            for i in range(n):
                step(i, outs[1, i], read[1, i], lambda: None)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(read[0], read[1])
    d.ok()


def test_a_plans_first_call_captured():
    """Nothing of a plan is made in a way that a capture forbids; graphs of a plan each may run side by side."""
    graphs, ds, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    for s, n in enumerate((1, 4, 60)):
        d = Device(Batch4([n, n], [900, 300], 8, 2, 128, BF16, seed=s))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d.attend()
        graphs.append(graph), ds.append(d)
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    for d in ds:
        d.ok()
        d.check()


def test_two_plans_on_two_streams():
    ds = [Device(Batch4([1] * 4 + [90], [2000, 30, 700, 1, 500], 8, 2, 128, BF16, seed=s)) for s in (1, 2)]
    ds += [Device(Batch4([1] * 4, [2000, 30, 700, 1], 16, 2, 64, F16, seed=s)) for s in (3, 4)]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(ds, streams):
            d.attend(stream=s)
    for d in ds:
        d.ok()
        d.check()


# ------------------------------------------------------------------ refusals and device errors
def test_refused_arguments():
    d = Device(Batch4([1, 20], [40, 20], 8, 2, 128, BF16))
    p, b = d.plan, d.batch
    k_out = torch.zeros(21, 2, 128, dtype=BF16, device="cuda")
    for call in (lambda: cs.cs_kv4_attention(p, b, d.q.float(), d.k, d.v, d.out),
                 lambda: cs.cs_kv4_attention(p, b, d.q, (d.k[0][:1], d.k[1]), d.v, d.out),
                 lambda: cs.cs_kv4_attention(p, b, d.q, (d.k[0], d.k[1][:1]), d.v, d.out),
                 lambda: cs.cs_kv4_attention(p, b, d.q, d.k, (d.v[0].char(), d.v[1]), d.out),
                 lambda: cs.cs_kv4_attention(p, b, d.q, d.k, cuda((d.v[0].cpu(), d.v[1].cpu()))[::-1], d.out),
                 lambda: cs.cs_kv4_attention(p, b, d.q, (d.k[0].cpu(), d.k[1]), d.v, d.out),
                 lambda: cs.cs_kv4_attention(p, b, d.q, d.k, d.v, d.out, lse=d.lse.double()),
                 lambda: cs.cs_kv4_read(p, b, d.k, d.v, k_out[:5], None), lambda: cs.cs_kv4_read(p, b, d.k, d.v, k_out.half(), None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        cs.cs_kv4_attention(p, b, d.q, d.k[0], d.v, d.out)
    with pytest.raises(TypeError):
        cs.cs_kv4_read(p, b, None, d.v, k_out, None)

    def refused(f, *a, status=cs.CS_ERR_INVALID_ARG, **k):
        with pytest.raises(cs.CSError) as e:
            f(*a, **k)
        assert e.value.status == status

    refused(cs.cs_kv4_attention, p, b, d.q, d.k, d.v, d.q)  # out is q
    refused(cs.cs_kv4_attention_shared, p, b, d.q, d.k, d.v, d.prefix_pages, 0, d.out)  # not asked for
    refused(cs.cs_kv4_read, p, b, d.k, d.v, None, None)
    refused(cs.cs_kv4_read, p, b, d.k, d.v, k_out, k_out)
    over = d.k[0].flatten()[:21 * 512].view(BF16).view(21, 256)
    refused(cs.cs_kv4_read, p, b, d.k, d.v, over, None)
    qkv = torch.zeros(21, 12 * 128, dtype=BF16, device="cuda")
    refused(cs.cs_kv4_append, p, b, qkv, d.out, d.k, d.k)
    refused(cs.cs_kv4_append, p, b, qkv, d.out, d.k, (d.v[0], d.k[1]))
    with cs.cs_kv_plan(d.b.desc(cs, rotary_dim=64)) as turning:
        tb = cs.cs_kv_batch(turning, d.cu_q, d.kv, d.table, tokens=21, max_q=20)
        refused(cs.cs_kv4_append, turning, tb, qkv, d.out, d.k, d.v)  # no table
        rope = rope_table(50, 64).cuda()
        refused(cs.cs_kv4_append, turning, tb, qkv, qkv[:, 128:128 + 1024], d.k, d.v, rope=rope)
        with pytest.raises(ValueError):
            cs.cs_kv4_append(turning, tb, qkv, d.out, d.k, d.v, rope=rope[:, :32])
    d.attend()
    d.ok()
    d.check()


def test_nothing_to_do():
    for q, kv, pad in (([0, 0], [5, 0], 4), ([0], [5], 0)):
        d = Device(Batch4(q, kv, 8, 2, 128, BF16, pad=pad))
        before = [x.clone() for x in (*d.k, *d.v)]
        out = torch.full((pad, 2, 128), 7.0, dtype=BF16, device="cuda")
        d.attend()
        cs.cs_kv4_append(d.plan, d.batch, torch.zeros(pad, 12 * 128, dtype=BF16, device="cuda"), d.out, d.k, d.v)
        cs.cs_kv4_read(d.plan, d.batch, d.k, d.v, out, torch.full_like(out, 7.0))
        d.ok()
        assert (d.out == 7).all() and (out == 7).all()
        assert all(torch.equal(x, y) for x, y in zip(before, (*d.k, *d.v)))


@pytest.mark.parametrize("n", [1, 3, 40])
def test_lengths_and_pages_that_do_not_fit(n):
    """Reported by the status, answered by CS_ERR_NEEDS_RESET, cleared by a reset; the other sequences are right."""
    def fresh():
        return Device(Batch4([n, n], [100, 90], 8, 2, 128, BF16, poison=False))

    for spoil in (lambda d: d.kv.__setitem__(0, 17 * 16 + 1000), lambda d: d.kv.__setitem__(0, -1),
                  lambda d: d.cu_q.__setitem__(0, n + 5), lambda d: d.cu_q.__setitem__(0, -3),
                  lambda d: d.table.__setitem__((0, 5), -1), lambda d: d.table.__setitem__((0, 2), BAD_PAGE)):
        d = fresh()
        spoil(d)
        d.attend()
        torch.cuda.synchronize()
        assert cs.cs_kv_status(d.plan) == cs.CS_ERR_INVALID_ARG
        assert "sequence 0" in cs.cs_last_error_string()
        ref, _, bound = d.b.reference(list(range(n, 2 * n)))
        assert (np.abs(okv.to64(d.out)[n:] - ref) <= bound).all()
        with pytest.raises(cs.CSError) as e:
            d.attend()
        assert e.value.status == cs.CS_ERR_NEEDS_RESET
        with pytest.raises(cs.CSError) as e:
            cs.cs_kv4_read(d.plan, d.batch, d.k, d.v, torch.empty(2 * n, 2, 128, dtype=BF16, device="cuda"), None)
        assert e.value.status == cs.CS_ERR_NEEDS_RESET
        cs.cs_kv_reset(d.plan)
        good = fresh()
        for x in ("kv", "cu_q", "table"):
            getattr(d, x).copy_(getattr(good, x))
        d.attend()
        d.ok()
        d.check()


def test_append_and_read_report_bad_pages_and_positions():
    for spoil in ("page", "position"):
        b = Batch4([1, 1], [30, 40], 8, 2, 128, BF16, poison=False)
        d = Device(b, rotary_dim=128)
        if spoil == "page":
            d.table[1, 2] = d.b.num_pages
        rows = 35 if spoil == "position" else 60
        qkv = torch.ones(2, 12 * 128, dtype=BF16, device="cuda")
        before = d.k[0].clone()
        cs.cs_kv4_append(d.plan, d.batch, qkv, d.out, d.k, d.v, rope=rope_table(rows, 128).cuda())
        torch.cuda.synchronize()
        assert cs.cs_kv_status(d.plan) == cs.CS_ERR_INVALID_ARG
        assert ("page" if spoil == "page" else "token 1") in cs.cs_last_error_string()
        changed = (d.k[0] != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(b.table[0, 29 // 16])]
        if spoil == "page":
            cs.cs_kv_reset(d.plan)
            out = torch.full((2, 2, 128), 7.0, dtype=BF16, device="cuda")
            cs.cs_kv4_read(d.plan, d.batch, d.k, d.v, None, out)
            torch.cuda.synchronize()
            assert cs.cs_kv_status(d.plan) == cs.CS_ERR_INVALID_ARG
            # the scale nearest to 1 / 7 is 0.140625, and 7 of it are held for 1
            assert (out[0] == 0.984375).all() and (out[1] == 7).all()


def test_a_cache_of_more_than_2_to_32_bytes():
    """Offsets behind 2^32 bytes of codes (2^33 values)."""
    pages = (1 << 32) // (64 * 8 * 64) + 40  # 64-position pages of 8 heads of 128
    b = Batch4([1, 70], [130, 200], 16, 8, 128, BF16, page_size=64)
    small = Device(b)
    plan = cs.cs_kv_plan(b.desc(cs, num_pages=pages))
    codes, scales = cs.cs_kv4_shapes(plan)
    k, v = ((torch.empty(codes, dtype=torch.uint8, device="cuda"), torch.empty(scales, dtype=torch.uint8, device="cuda")) for _ in range(2))
    far = b.table.clone()
    for i, page in enumerate(b.table.flatten().tolist()):
        if page != BAD_PAGE:
            far.view(-1)[i] = pages - 1 - page
            for to, of in ((k, small.k), (v, small.v)):
                for x, y in zip(to, of):
                    x[pages - 1 - page] = y[page]
    for tokens, max_q in ((71, 70), (2, 1)):
        cu = small.cu_q if tokens == 71 else torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        batch = cs.cs_kv_batch(plan, cu, small.kv, far.cuda(), tokens=tokens, max_q=max_q)
        near = cs.cs_kv_batch(small.plan, cu, small.kv, small.table, tokens=tokens, max_q=max_q)
        q = small.q[:tokens].contiguous()
        outs = [torch.zeros(tokens, 16, 128, dtype=BF16, device="cuda") for _ in range(2)]
        cs.cs_kv4_attention(plan, batch, q, k, v, outs[0])
        cs.cs_kv4_attention(small.plan, near, q, small.k, small.v, outs[1])
        torch.cuda.synchronize()
        assert cs.cs_kv_status(plan) == cs.CS_OK and torch.equal(outs[0], outs[1])
        qkv = torch.randn(tokens, 32 * 128, device="cuda").to(BF16)
        for p, bt, kk, vv in ((plan, batch, k, v), (small.plan, near, small.k, small.v)):
            cs.cs_kv4_append(p, bt, qkv, torch.zeros_like(outs[0]), kk, vv)
        reads = [torch.zeros(2, tokens, 8, 128, dtype=BF16, device="cuda") for _ in range(2)]
        cs.cs_kv4_read(plan, batch, k, v, reads[0][0], reads[0][1])
        cs.cs_kv4_read(small.plan, near, small.k, small.v, reads[1][0], reads[1][1])
        torch.cuda.synchronize()
        assert cs.cs_kv_status(plan) == cs.CS_OK and torch.equal(reads[0], reads[1])
        assert np.array_equal(okv.to64(reads[0][0]), o4.held(qkv.view(tokens, 32, 128)[:, 16:24].cpu()))
