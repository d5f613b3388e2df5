"""The paged cache operators on the GPU against the float64 definitions."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import consumer_gemm_chain_gb300 as cs
import oracle
from kv_util import BAD_PAGE, Batch, rope_table
from oracle import kv as okv

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Device:
    """A test batch on the GPU, with its plan."""

    def __init__(self, b: Batch, **desc):
        self.b = b
        self.plan = cs.cs_kv_plan(b.desc(cs, **desc))
        self.cu_q, self.kv, self.table = b.cu_q.cuda(), b.kv.cuda(), b.table.cuda()
        self.q, self.kc, self.vc, self.prefix_pages = b.q.cuda(), b.kc.cuda(), b.vc.cuda(), b.prefix_pages.cuda()
        self.batch = cs.cs_kv_batch(self.plan, self.cu_q, self.kv, self.table, tokens=b.tokens, max_q=b.max_q)
        self.out = torch.full((b.tokens, b.heads, b.head_dim), 7.0, dtype=b.dtype, device="cuda")
        self.lse = torch.full((b.tokens, b.heads), 7.0, device="cuda")

    def attend(self, q=None, out=None, lse=True, stream=None):
        q, out = self.q if q is None else q, self.out if out is None else out
        lse = self.lse if lse else None
        if self.b.prefix:
            cs.cs_kv_attention_shared(self.plan, self.batch, q, self.kc, self.vc, self.prefix_pages, self.b.prefix, out, lse,
                                      stream=stream)
        else:
            cs.cs_kv_attention(self.plan, self.batch, q, self.kc, self.vc, out, lse, stream=stream)

    def ok(self):
        torch.cuda.synchronize()
        st = cs.cs_kv_status(self.plan)
        assert st == cs.CS_OK, f"{cs.STATUS_NAMES.get(st)}: {cs.cs_last_error_string()}"

    def check(self, tokens=None, out=None):
        """The outputs against the reference (rows `tokens`, default all), the padding untouched."""
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


HEADS = [(128, 1, 64), (100, 1, 128), (12, 12, 128), (8, 2, 64), (28, 4, 128), (16, 1, 64), (6, 2, 128), (40, 2, 64)]


@pytest.mark.parametrize("heads,kv_heads,head_dim", HEADS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("q,kv", [
    ([1], [1]), ([1], [2000]), ([1, 1, 0, 1], [17, 128, 5, 129]), ([4, 0, 1], [4, 0, 300]), ([5, 3], [700, 3]),
    ([130, 1, 33], [130, 257, 64]), ([257], [400])])
def test_attention(heads, kv_heads, head_dim, dtype, q, kv):
    run(Batch(q, kv, heads, kv_heads, head_dim, dtype, pad=2, seed=len(q) + heads))


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("q,kv", [([1, 1], [333, 15]), ([150, 7], [333, 200])])
def test_pages_and_layouts(page_size, layout, q, kv):
    for heads, head_dim, dtype in ((8, 128, BF16), (8, 64, F16)):
        run(Batch(q, kv, heads, 2, head_dim, dtype, page_size=page_size, layout=layout, seed=page_size))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 128), (129, 130), (1000, 5), (37, 1000)])
@pytest.mark.parametrize("q,kv", [([1, 1, 1], [900, 37, 140]), ([3, 300, 64], [500, 400, 901])])
def test_window_and_sinks(window, sinks, q, kv):
    run(Batch(q, kv, 8, 2, 128, BF16, window=window, sinks=sinks, seed=window))
    run(Batch(q, kv, 6, 6, 64, F16, window=window, sinks=sinks, seed=window, page_size=128, layout="head"))


@pytest.mark.parametrize("heads,kv_heads,head_dim,q,kv,window,sinks", [
    (12, 12, 128, [2226, 1517], [2226, 1517], 1024, 4), (8, 2, 64, [1900, 700, 1], [2500, 700, 3000], 700, 130),
    (12, 4, 128, [3000], [3000], 0, 0), (16, 1, 128, [640], [5000], 2000, 1)])
def test_many_items(heads, kv_heads, head_dim, q, kv, window, sinks):
    """More items than SMs, cut at places that depend on windows and sinks: rows at the
    borders of tiles and items, and some between."""
    b = Batch(q, kv, heads, kv_heads, head_dim, F16, window=window, sinks=sinks, seed=window)
    d = Device(b)
    d.attend()
    d.ok()
    rows, at = [], 0
    for n in q:
        rows += [at + i for i in range(n) if i % 128 in (0, 127) or i % 85 == 84]
        at += n
    d.check(rows)


@pytest.mark.parametrize("q,kv,prefix", [([1] * 40, [1 + 9 * i for i in range(40)], 3001), ([1, 3, 2], [400, 90, 2], 700),
                                         ([1], [200], 40), ([90, 1], [300, 20], 1000)])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_right_behind_one_another(q, kv, prefix, captured):
    """Kernels start while the ones before them end: the same results, bit by bit, as with
    nothing else running (append, attention behind a prefix, attention; again with other queries)."""
    b = Batch(q, kv, 8, 2, 128, BF16, prefix=prefix, seed=prefix)
    d = Device(b, rotary_dim=0)
    g = torch.Generator().manual_seed(5)
    n = 6
    qkv = (torch.randn(n, b.tokens, 12 * 128, generator=g)).to(BF16).cuda()
    outs = torch.zeros(2, n, 2, b.tokens, 8, 128, dtype=BF16, device="cuda")
    qs = torch.zeros(2, b.tokens, 8, 128, dtype=BF16, device="cuda")

    def step(i, out, pause):
        cs.cs_kv_append(d.plan, d.batch, qkv[i], qs[i % 2], d.kc, d.vc)
        pause()
        cs.cs_kv_attention_shared(d.plan, d.batch, qs[i % 2], d.kc, d.vc, d.prefix_pages, b.prefix, out[0])
        pause()
        cs.cs_kv_attention(d.plan, d.batch, qs[i % 2], d.kc, d.vc, out[1])
        pause()

    for i in range(n):
        step(i, outs[0, i], torch.cuda.synchronize)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(n):
                step(i, outs[1, i], lambda: None)
        for _ in range(3):
            outs[1].fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[0], outs[1])
    else:
        for _ in range(3):
            outs[1].fill_(7)
            for i in range(n):
                step(i, outs[1, i], lambda: None)
            torch.cuda.synchronize()
            assert torch.equal(outs[0], outs[1])
    d.ok()


@pytest.mark.parametrize("heads,kv_heads,head_dim,q,kv,window,sinks", [
    (8, 2, 128, [600, 1, 70], [6000, 3900, 4100], 0, 0), (8, 8, 64, [600, 70, 0, 1], [6000, 4100, 0, 3900], 3400, 130),
    (12, 12, 64, [700, 900], [5000, 7000], 0, 0), (16, 1, 128, [40, 300], [9000, 4000], 3300, 4)])
@pytest.mark.parametrize("num_sms", [0, 37])
def test_long_items(heads, kv_heads, head_dim, q, kv, window, sinks, num_sms):
    """Items long enough to be cut and joined, and shorter ones between them."""
    b = Batch(q, kv, heads, kv_heads, head_dim, BF16, window=window, sinks=sinks, seed=kv[0], page_size=64)
    d = Device(b, num_sms=num_sms)
    d.attend()
    d.ok()
    rows, at = [], 0
    for n in q:
        rows += [at + i for i in range(n) if i % 64 in (0, 63) or i == n - 1]
        at += n
    d.check(rows)


@pytest.mark.parametrize("lens", [[512] * 6, [300] * 7, [1024, 90, 700, 2, 511], [256], [20] * 90])
def test_whole_items(lens):
    """Prompts short enough for no item to be cut: about as many items as SMs, fewer and more."""
    b = Batch(lens, lens, 12, 12, 128, F16, seed=len(lens))
    d = Device(b)
    for _ in range(2):
        d.out.fill_(7), d.lse.fill_(7)
        d.attend()
    d.ok()
    rows, at = [], 0
    for n in lens:
        rows += [at + i for i in range(n) if i % 128 in (0, 127) or i == n - 1]
        at += n
    d.check(rows)


@pytest.mark.parametrize("prefix", [1, 16, 127, 500, 2049])
@pytest.mark.parametrize("q,kv", [([1] * 5, [1, 40, 130, 2, 16]), ([1, 0, 3], [9, 0, 3]), ([40, 1, 70], [40, 300, 75]), ([2], [1])])
def test_shared_prefix(prefix, q, kv):
    run(Batch(q, kv, 8, 2, 128, BF16, prefix=prefix, pad=3, seed=prefix))
    run(Batch(q, kv, 7, 1, 64, F16, prefix=prefix, page_size=64, layout="head", seed=prefix))


def test_tokens_before_position_zero():
    for q, kv in (([4, 3], [2, 0]), ([200, 1], [60, 0])):
        d = run(Batch(q, kv, 8, 2, 128, BF16))
        assert (d.out[:q[0] - kv[0]] == 0).all()
        run(Batch(q, kv, 4, 4, 64, F16, window=8, sinks=2))


@pytest.mark.parametrize("q,kv,rows", [([1, 1], [40000, 9000], None), ([700, 1], [9001, 5000], [0, 1, 350, 699, 700]),
                                       ([3], [30001], None), ([2500], [2500], [0, 1, 127, 128, 1300, 2498, 2499])])
def test_long_contexts(q, kv, rows):
    b = Batch(q, kv, 8, 2, 128, BF16, page_size=64, seed=3)
    d = Device(b)
    d.attend()
    d.ok()
    d.check(rows)


def test_many_sequences():
    run(Batch([1] * 3001, [5] * 3000 + [40], 2, 1, 64, F16))
    run(Batch([0, 1] * 900, [3, 4] * 900, 2, 2, 64, BF16, poison=False))
    run(Batch([1] * 99 + [30], [7] * 99 + [64], 4, 2, 64, F16))
    r = np.random.default_rng(0)
    kv = [int(x) for x in r.integers(1, 90, 700)]
    run(Batch([1] * 700, kv, 4, 2, 64, F16))
    q = [int(x) for x in r.integers(0, 9, 300)]
    run(Batch(q, [n + int(x) for n, x in zip(q, r.integers(0, 60, 300))], 4, 2, 64, BF16))


@pytest.mark.parametrize("window", [0, 600])
def test_a_value_that_is_not_finite_and_seen_by_many_rows(window):
    """Rows that see it have it in their results, and no others; the call takes about as long
    as without it (not as if every one of those rows had been computed again)."""
    b = Batch([4096], [4096], 16, 4, 64, F16, window=window, seed=window)
    d = Device(b)
    d.attend()
    d.ok()
    clean = d.out.clone()
    page, slot = int(b.table[0, 2000 // 16]), 2000 % 16
    d.vc[page, slot, :, 3] = math.inf
    a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    d.attend()
    e.record()
    d.ok()
    assert a.elapsed_time(e) < 20.0
    sees = torch.zeros(4096, dtype=torch.bool, device="cuda")
    sees[2000:2000 + window if window else None] = True
    assert not torch.isfinite(d.out[sees][:, :, 3]).any()
    d.out[sees, :, 3] = clean[sees, :, 3]
    rows = [*range(1980, 2004), *range(2590, 2606), 100, 1900, 2300, 4095]
    d.check(rows)
    assert torch.equal(d.out[:1900], clean[:1900])


def test_values_that_are_not_finite_in_the_other_half_of_a_short_item():
    """Items of one row tile whose key tiles go to two halves in turn, none of them cut:
    the spoilt key lies in the second half's tile."""
    b = Batch([5] * 60, [250] * 60, 8, 2, 128, BF16, seed=3)
    for s in range(60):
        page, slot = int(b.table[s, 249 // 16]), 249 % 16
        b.vc[page, slot, :, 5:9] = math.nan
        b.v[s][249, :, 5:9] = 0.0  # rows that do not see it never read it
    d = Device(b)
    d.attend()
    d.ok()
    ref, _, bound = b.reference()
    got = okv.to64(d.out)
    for t in range(300):
        ok = np.ones(128, dtype=bool)
        ok[5:9] = t % 5 < 4
        assert (np.abs(got[t, :, ok] - ref[t, :, ok]) <= bound[t, :, ok]).all(), t
        assert t % 5 < 4 or not np.isfinite(got[t, :, 5:9]).any(), t


@pytest.mark.parametrize("q,kv", [([4, 1], [70, 9]), ([3], [900]), ([200, 30], [300, 30]), ([130], [2000])])
@pytest.mark.parametrize("window,prefix", [(0, 0), (33, 0), (0, 50)])
def test_values_that_are_not_finite_at_keys_hidden_from_some_rows(q, kv, window, prefix):
    """NaN and infinities at keys that only later tokens (or, under a window, only earlier
    ones) see: every other row is as if they were not there, and those rows are NaN."""
    for dtype, bad in ((BF16, math.nan), (F16, math.inf)):
        b = Batch(q, kv, 8, 2, 128, dtype, window=window, sinks=2 if window else 0, prefix=prefix, seed=kv[0])
        spoilt = []  # (sequence, key): seen by the last token only, and by the first only
        for s, (n, m) in enumerate(zip(q, kv)):
            spoilt.append((s, m - 1))
            if window and m - n - window + 1 >= 2 and n > 1:
                spoilt.append((s, m - n - window + 1))
        for s, j in spoilt:
            page, slot = int(b.table[s, j // 16]), j % 16
            b.vc[page, slot, :, 5:9] = bad
            b.v[s][j, :, 5:9] = 0.0  # rows that do not see it never read it
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
                ok[5:9] = not hit
                assert (np.abs(got[t, :, ok] - ref[t, :, ok]) <= bound[t, :, ok]).all(), (s, i)
                assert not hit or not np.isfinite(got[t, :, 5:9]).any(), (s, i)
                t += 1


@pytest.mark.parametrize("q,kv", [([4], [70]), ([200], [300])])
def test_keys_that_are_not_finite_where_hidden(q, kv):
    b = Batch(q, kv, 8, 2, 64, BF16)
    n, m = q[0], kv[0]
    page, slot = int(b.table[0, (m - 1) // 16]), (m - 1) % 16
    b.kc[page, slot] = math.nan
    d = Device(b)
    d.attend()
    d.ok()
    ref, _, bound = b.reference(list(range(n - 1)))
    got = okv.to64(d.out)
    assert (np.abs(got[:n - 1] - ref) <= bound).all() and np.isnan(got[n - 1]).all()


def test_large_scores():
    """Rows whose maximum keeps rising by much, and weights far below the row's largest."""
    for n in (1, 200):
        b = Batch([n], [600], 4, 2, 128, BF16, spread=1.0, scale=1.0, seed=5)
        b.k[0] = (b.k[0].float() * torch.linspace(0.02, 3, 600)[:, None, None]).to(BF16)
        b2 = Batch([n], [600], 4, 2, 128, BF16, scale=1.0, seed=5)
        # the cache of b2 with b's keys
        for j in range(600):
            b2.kc[b2.table[0, j // 16], j % 16] = b.k[0][j]
        b2.k = b.k
        d = Device(b2)
        d.attend()
        d.ok()
        ref, lse, bound = b2.reference()
        got = okv.to64(d.out)
        # scores reach 3 * 128 * 4 in sum: 128 products in 32 bits are off by up to
        # 2^-24 * 128 * sum|q k| scale, both in a weight and in the row's sum
        worst = 2 * 2.0 ** -24 * 128 * float((b2.q.float().abs().amax() * b2.k[0].float().abs().amax() * 128))
        assert (np.abs(got - ref) <= bound * (1 + worst / 2.0 ** -11)).all()


def test_rows_of_other_strides():
    b = Batch([1, 90, 3], [50, 90, 700], 8, 2, 128, BF16, pad=2)
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
    for b in (Batch([1] * 9, [900, 5, 77, 3000, 1, 128, 129, 2000, 64], 16, 2, 128, BF16),
              Batch([300, 1, 50], [900, 3000, 50], 8, 2, 64, F16, prefix=0),
              Batch([1] * 20, list(range(1, 21)), 8, 2, 128, BF16, prefix=1000)):
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
        d = Device(Batch([1, 60], [300, 700], 8, 2, 128, BF16), num_sms=sms)
        d.attend()
        d.ok()
        d.check()
        d.out.fill_(7)
        d.attend(lse=False)
        d.ok()
        d.check()


def test_a_captured_step_with_other_lengths():
    """Append and attention captured once, replayed as a sequence grows."""
    heads, hk, d = 8, 2, 128
    for n in (1, 20):
        full = Batch([n, n], [300 + n, 70 + n], heads, hk, d, BF16, poison=False, seed=n)
        dev = Device(full)
        qkv = torch.cat([full.q.flatten(1), torch.cat([k[-n:].flatten(1) for k in full.k]),
                         torch.cat([v[-n:].flatten(1) for v in full.v])], 1).cuda()
        want = dev.kc.clone(), dev.vc.clone()
        # the cache before the step; the rotation is off
        for s, m in enumerate(full.kv_lens):
            for j in range(m - n, m):
                for c in (dev.kc, dev.vc):
                    c[full.table[s, j // 16], j % 16] = 9
        before = dev.kc.clone(), dev.vc.clone()
        q_out = torch.zeros_like(dev.q)

        def step():
            cs.cs_kv_append(dev.plan, dev.batch, qkv, q_out, dev.kc, dev.vc)
            cs.cs_kv_attention(dev.plan, dev.batch, q_out, dev.kc, dev.vc, dev.out, dev.lse)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        short = torch.tensor([40, 20 + n], dtype=torch.int32, device="cuda")
        dev.kv.copy_(short)
        with torch.cuda.graph(graph):
            step()
        graph.replay()
        dev.ok()
        dev.kv.copy_(full.kv)
        dev.kc.copy_(before[0]), dev.vc.copy_(before[1])
        dev.out.fill_(7), dev.lse.fill_(7)
        graph.replay()
        dev.ok()
        assert torch.equal(dev.kc, want[0]) and torch.equal(dev.vc, want[1])
        dev.check()


def test_two_plans_on_two_streams():
    ds = [Device(Batch([1] * 4 + [90], [2000, 30, 700, 1, 500], 8, 2, 128, BF16, seed=s)) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(ds, streams):
            d.attend(stream=s)
    for d in ds:
        d.ok()
        d.check()


# ------------------------------------------------------------------ append
def append_case(q, kv, heads, hk, d, dtype, rotary, pairing, layout, page_size, pad=0, in_place=False, positions=False, shift=0):
    b = Batch(q, kv, heads, hk, d, dtype, page_size=page_size, layout=layout, pad=pad, seed=rotary + d)
    dev = Device(b, rotary_dim=rotary, rotary_pairing=pairing)
    g = torch.Generator().manual_seed(9)
    width = (heads + 2 * hk) * d
    store = torch.randn(b.tokens, width + shift, generator=g).to(dtype)
    qkv = store[:, :width]
    rows = max(kv) + 50
    rope = rope_table(rows, rotary) if rotary else None
    pos_of, where = [], []
    for s, (n, m) in enumerate(zip(q, kv)):
        pos_of += list(range(m - n, m))
        where += [(s, p) for p in range(m - n, m)]
    ids = torch.randint(0, rows, (b.tokens,), generator=g, dtype=torch.int32) if positions else None
    kc0, vc0 = dev.kc.clone(), dev.vc.clone()
    dstore = store.cuda()
    dqkv = dstore[:, :width]
    q_out = dqkv[:, :heads * d] if in_place else torch.full((b.tokens, heads, d), 7.0, dtype=dtype, device="cuda")
    cs.cs_kv_append(dev.plan, dev.batch, dqkv, q_out, dev.kc, dev.vc, rope=None if rope is None else rope.cuda(),
                    positions=None if ids is None else ids.cuda())
    dev.ok()
    x = okv.to64(qkv).reshape(b.tokens, heads + 2 * hk, d)
    angles = ids.numpy() if positions else np.maximum(np.array(pos_of + [0] * pad), 0)
    y, size = x.copy(), np.abs(x)
    if rotary:
        t = okv.to64(rope)[angles][:, None]
        qk = slice(0, heads + hk)
        y[:, qk] = okv.rotate(x[:, qk], t[..., :rotary // 2], t[..., rotary // 2:], pairing)
        size[:, qk] = okv.rotate(np.abs(x[:, qk]), np.abs(t[..., :rotary // 2]), -np.abs(t[..., rotary // 2:]), pairing)
        size[:, qk] = np.maximum(np.abs(size[:, qk]), np.abs(x[:, qk]).max())
    # two products and their sum in 32 bits (3 * 2^-24 of the terms' sizes), one rounding
    u = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * u
    bound = u * np.abs(y) + (1 + u) * 3 * 2.0 ** -24 * 2 * size + tiny
    got_q = okv.to64(q_out).reshape(b.tokens, heads, d)
    live = [i for i, p in enumerate(pos_of) if p >= 0]
    assert (np.abs(got_q[live] - y[live, :heads]) <= bound[live, :heads]).all()
    if in_place:
        assert torch.equal(dstore[:, heads * d:].cpu(), store[:, heads * d:])
        assert torch.equal(dstore[b.real:].cpu(), store[b.real:])
    else:
        assert (q_out[b.real:] == 7).all()
    kc, vc = dev.kc.cpu(), dev.vc.cpu()
    kc0, vc0 = kc0.cpu(), vc0.cpu()
    for i in live:
        s, p = where[i]
        page, slot = int(b.table[s, p // page_size]), p % page_size
        at = (page, slot) if layout == "token" else (page, slice(None), slot)
        assert (np.abs(okv.to64(kc[at]) - y[i, heads:heads + hk]) <= bound[i, heads:heads + hk]).all()
        assert torch.equal(vc[at], qkv[i].reshape(-1, d)[heads + hk:])
        kc[at], vc[at] = kc0[at], vc0[at]
    assert torch.equal(kc.view(torch.int16), kc0.view(torch.int16)) and torch.equal(vc.view(torch.int16), vc0.view(torch.int16))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,hk,d,rotary,pairing", [
    (12, 12, 128, 128, "half"), (8, 2, 64, 64, "adjacent"), (28, 4, 128, 32, "half"), (6, 1, 64, 16, "adjacent"),
    (5, 5, 128, 112, "half"), (4, 2, 64, 0, "half")])
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


def test_append_leaves_out_tokens_before_position_zero():
    append_case([5, 2], [3, 0], 8, 2, 64, F16, 64, "half", "token", 16)


# ------------------------------------------------------------------ together
def test_prompt_then_tokens_through_an_attention_chain():
    """A prompt and then single tokens through cs_attn_cached_forward: every step's rows
    equal the whole sequence's attention layer."""
    H, heads, dtype = 256, 2, F16
    F, total, prompt = heads * 128, 40, 33
    g = torch.Generator().manual_seed(4)
    X = (torch.randn(total, H, generator=g) * 0.5).to(dtype)
    Wqkv = (torch.randn(H, 3 * F, generator=g) * 0.06).to(dtype)
    Wo = (torch.randn(F, H, generator=g) * 0.06).to(dtype)
    rope = rope_table(total, 128)
    X64, t = okv.to64(X), okv.to64(rope)[:, None]
    qkv = (X64 @ okv.to64(Wqkv)).reshape(total, 3 * heads, 128)
    qk = okv.rotate(qkv[:, :2 * heads], t[..., :64], t[..., 64:], "half")
    O = np.zeros((total, heads, 128))
    for p in range(total):
        for h in range(heads):
            O[p, h] = okv.attend(qk[p, h], qk[:, heads + h], qkv[:, 2 * heads + h], okv.visible(p, total, 0, 0), 128 ** -0.5)[0]
    ref = O.reshape(total, F) @ okv.to64(Wo)
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=heads, num_pages=4, max_tokens=prompt, max_seqs=1,
                                            rotary_dim=128))
    kc, vc = (torch.full(plan.cache_shape, math.nan, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    done = 0
    for n in [prompt] + [1] * (total - prompt):
        desc = cs.cs_chain_desc_init(kind="attn", M=n, H=H, F=F, dtype=dtype, heads=heads, head_dim=128, split_k=1, sk_tiles=-1)
        with cs.cs_chain_plan(desc) as chain:
            batch = cs.cs_kv_batch(plan, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                   torch.tensor([done + n], dtype=torch.int32, device="cuda"), table, tokens=n, max_q=n)
            Y = torch.empty(n, H, dtype=dtype, device="cuda")
            for _ in range(2):  # a step may be run again
                cs.cs_attn_cached_forward(chain, plan, batch, X[done:done + n].cuda(), Wqkv.cuda(), Wo.cuda(), Y, kc, vc,
                                          rope=rope.cuda())
            torch.cuda.synchronize()
            assert cs.cs_chain_status(chain) == cs.CS_OK and cs.cs_kv_status(plan) == cs.CS_OK
            assert oracle.rel_err(Y.cpu(), ref[done:done + n]) <= 5e-3
        done += n


def test_a_run_of_steps():
    """Prompts and then single tokens of three sequences, appended and attended with a
    window, against the definition over everything appended."""
    heads, hk, d, window, sinks, dtype = 8, 2, 64, 50, 3, BF16
    r = np.random.default_rng(2)
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=hk, head_dim=d, page_size=16, num_pages=40,
                                            max_tokens=300, max_seqs=3, rotary_dim=32, window=window, sinks=sinks))
    kc, vc = (torch.full(plan.cache_shape, math.nan, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.from_numpy(r.permutation(40)[:36].reshape(3, 12).astype(np.int32)).cuda()
    rope = rope_table(200, 32)
    lens, keys, vals = [0, 0, 0], [[], [], []], [[], [], []]
    t64 = okv.to64(rope)
    for step in ([100, 1, 0], [1, 0, 130], [1, 1, 1], [20, 3, 1], [1, 1, 1]):
        lens = [m + n for m, n in zip(lens, step)]
        T = sum(step)
        qkv = torch.from_numpy(r.standard_normal((T, (heads + 2 * hk) * d))).to(dtype)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(step)]), dtype=torch.int32, device="cuda")
        batch = cs.cs_kv_batch(plan, cu, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, tokens=T, max_q=max(step))
        work = qkv.cuda()
        out = torch.empty(T, heads, d, dtype=dtype, device="cuda")
        cs.cs_kv_append(plan, batch, work, work[:, :heads * d], kc, vc, rope=rope.cuda())
        cs.cs_kv_attention(plan, batch, work[:, :heads * d], kc, vc, out)
        torch.cuda.synchronize()
        assert cs.cs_kv_status(plan) == cs.CS_OK
        got, i = okv.to64(out), 0
        rotated = okv.to64(work).reshape(T, heads + 2 * hk, d)[:, :heads]  # the queries as stored
        x = okv.to64(qkv).reshape(T, heads + 2 * hk, d)
        for s, n in enumerate(step):
            for p in range(lens[s] - n, lens[s]):
                keys[s].append(okv.rotate(x[i + p - lens[s] + n, heads:heads + hk], t64[p, :16], t64[p, 16:], "half"))
                vals[s].append(x[i + p - lens[s] + n, heads + hk:])
            for p in range(lens[s] - n, lens[s]):
                seen = okv.visible(p, lens[s], window, sinks)
                for h in range(heads):
                    k = np.array([y[h // 4] for y in keys[s]])
                    k = okv.to64(torch.from_numpy(k).to(dtype))  # the cache holds the rounded keys
                    o, _, a = okv.attend(rotated[i, h], k, np.array([y[h // 4] for y in vals[s]]), seen, d ** -0.5)
                    # weights and output rounded (2^-8 each); a key that 32-bit and 64-bit rotation
                    # round apart is off by 2^-7 of itself, its score by 2^-7 |q_i k_i| / 8 <= 2^-6
                    assert (np.abs(got[i, h] - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -6) * a + 1e-6).all()
                i += 1


# ------------------------------------------------------------------ refusals and device errors
def test_refused_arguments():
    d = Device(Batch([1, 20], [40, 20], 8, 2, 128, BF16, prefix=0))
    p, b = d.plan, d.batch
    with pytest.raises(ValueError):
        cs.cs_kv_attention(p, b, d.q.float(), d.kc, d.vc, d.out)
    with pytest.raises(ValueError):
        cs.cs_kv_attention(p, b, d.q[:5], d.kc, d.vc, d.out)
    with pytest.raises(ValueError):
        cs.cs_kv_attention(p, b, d.q, d.kc[:1], d.vc, d.out)
    with pytest.raises(ValueError):
        cs.cs_kv_attention(p, b, d.q.cpu(), d.kc, d.vc, d.out)
    with pytest.raises(ValueError):
        cs.cs_kv_attention(p, b, d.q.transpose(0, 1).contiguous().transpose(0, 1), d.kc, d.vc, d.out)
    with pytest.raises(ValueError):
        cs.cs_kv_attention(p, b, d.q, d.kc, d.vc, d.out, lse=d.lse.double())
    with pytest.raises(ValueError):
        cs.cs_kv_batch(p, d.cu_q.long(), d.kv, d.table, tokens=21, max_q=20)
    with pytest.raises(ValueError):
        cs.cs_kv_batch(p, d.cu_q[:-1], d.kv, d.table, tokens=21, max_q=20)

    def refused(status, f, *a, **k):
        with pytest.raises(cs.CSError) as e:
            f(*a, **k)
        assert e.value.status == status

    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention, p, b, d.q, d.kc, d.vc, d.q)  # out is q
    both = torch.zeros(21, 2 * 1024, dtype=BF16, device="cuda")
    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention, p, b, both[:, :1024], d.kc, d.vc, both[:, 512:1536])
    cs.cs_kv_attention(p, b, both[:, :1024], d.kc, d.vc, both[:, 1024:])  # side by side
    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention_shared, p, b, d.q, d.kc, d.vc, d.prefix_pages, 0, d.out)  # not asked for
    big = cs.cs_kv_batch(p, d.cu_q, d.kv, d.table, tokens=22, max_q=20)
    q22 = torch.zeros(22, 8, 128, dtype=BF16, device="cuda")
    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention, p, big, q22, d.kc, d.vc, torch.zeros_like(q22))
    none = cs.cs_kv_batch(p, d.cu_q, d.kv, d.table, tokens=21, max_q=0)
    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention, p, none, d.q, d.kc, d.vc, d.out)
    odd = torch.zeros(21, 8 * 128 + 4, dtype=BF16, device="cuda")
    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention, p, b, odd[:, :1024], d.kc, d.vc, d.out)
    refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_attention, p, b, q22.flatten(1)[:, :1024].flatten()[4:4 + 1024 * 21].view(21, 1024),
            d.kc, d.vc, d.out)  # not 16-byte aligned
    with cs.cs_kv_plan(d.b.desc(cs, rotary_dim=64)) as turning:
        qkv = torch.zeros(21, 12 * 128, dtype=BF16, device="cuda")
        tb = cs.cs_kv_batch(turning, d.cu_q, d.kv, d.table, tokens=21, max_q=20)
        refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_append, turning, tb, qkv, d.out, d.kc, d.vc)  # no table
        rope = rope_table(50, 64).cuda()
        refused(cs.CS_ERR_INVALID_ARG, cs.cs_kv_append, turning, tb, qkv, qkv[:, 128:128 + 1024], d.kc, d.vc, rope=rope)
        with pytest.raises(ValueError):
            cs.cs_kv_append(turning, tb, qkv, d.out, d.kc, d.vc, rope=rope[:, :32])
    d.attend()
    d.ok()
    d.check()


def test_nothing_to_do():
    d = Device(Batch([0, 0], [5, 0], 8, 2, 128, BF16, pad=4))
    d.attend()
    d.ok()
    assert (d.out == 7).all()
    d = Device(Batch([0], [5], 8, 2, 128, BF16))
    d.attend()
    d.ok()


@pytest.mark.parametrize("n", [1, 40])
def test_lengths_and_pages_that_do_not_fit(n):
    """Reported by the status, answered by CS_ERR_NEEDS_RESET, cleared by a reset; the other sequences are right."""
    def fresh():
        return Device(Batch([n, n], [100, 90], 8, 2, 128, BF16, poison=False))

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
        cs.cs_kv_reset(d.plan)
        good = fresh()
        for x in ("kv", "cu_q", "table"):
            getattr(d, x).copy_(getattr(good, x))
        d.attend()
        d.ok()
        d.check()


def test_append_reports_bad_pages_and_positions():
    for spoil in ("page", "position"):
        b = Batch([1, 1], [30, 40], 8, 2, 128, BF16, poison=False)
        d = Device(b, rotary_dim=128)
        if spoil == "page":
            d.table[1, 2] = d.b.num_pages
        rows = 35 if spoil == "position" else 60
        qkv = torch.ones(2, 12 * 128, dtype=BF16, device="cuda")
        before = d.kc.clone()
        cs.cs_kv_append(d.plan, d.batch, qkv, d.out, d.kc, d.vc, rope=rope_table(rows, 128).cuda())
        torch.cuda.synchronize()
        assert cs.cs_kv_status(d.plan) == cs.CS_ERR_INVALID_ARG
        assert ("page" if spoil == "page" else "token 1") in cs.cs_last_error_string()
        changed = (d.kc != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(b.table[0, 29 // 16])]


def test_a_cache_of_more_than_2_to_31_elements():
    """Offsets behind 2^31 elements and 2^32 bytes."""
    pages = (1 << 31) // (64 * 8 * 128) + 40  # 64-position pages of 8 heads of 128
    b = Batch([1, 70], [130, 200], 16, 8, 128, BF16, page_size=64)
    plan = cs.cs_kv_plan(b.desc(cs, num_pages=pages))
    kc, vc = (torch.empty(plan.cache_shape, dtype=BF16, device="cuda") for _ in range(2))
    d = Device(b)
    far = b.table.clone()
    for i, page in enumerate(b.table.flatten().tolist()):
        if page != BAD_PAGE:
            far.view(-1)[i] = pages - 1 - page
            kc[pages - 1 - page], vc[pages - 1 - page] = d.kc[page], d.vc[page]
    batch = cs.cs_kv_batch(plan, d.cu_q, d.kv, far.cuda(), tokens=71, max_q=70)
    cs.cs_kv_attention(plan, batch, d.q, kc, vc, d.out, d.lse)
    torch.cuda.synchronize()
    assert cs.cs_kv_status(plan) == cs.CS_OK
    d.check()
    qkv = torch.randn(71, 32 * 128, device="cuda").to(BF16)
    cs.cs_kv_append(plan, batch, qkv, d.out, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[far[1, 3], 199 % 64], qkv[70].view(32, 128)[16:24])
    assert torch.equal(vc[far[0, 2], 129 % 64], qkv[0].view(32, 128)[24:])
