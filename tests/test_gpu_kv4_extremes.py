"""The paged cache in 4 bits on the GPU where numbers come near the ends of their types."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import consumer_gemm_chain_gb300 as cs
from kv4_util import Batch4, parts
from oracle import kv as okv
from oracle import kv4 as o4
from test_gpu_kv4 import Device

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def attend(q, k, v, dtype, **desc):
    """(out, lse) of the last len(q) tokens of one sequence over keys k and values v [keys, key heads, d], held as they are
    quantised or given as pairs of codes and scales; q [tokens, heads, d].  Pages of 16, TOKEN layout."""
    tokens, heads, d = q.shape
    keys, hk = len(k), k.shape[1]
    pages = -(-keys // 16)

    def cache(x):
        whole = torch.zeros(pages * 16, hk, d, dtype=torch.float64)
        whole[:keys] = x
        return tuple(y.cuda() for y in parts(whole.view(pages, 16, hk, d), "token"))

    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=hk, head_dim=d, num_pages=pages, max_tokens=tokens,
                                            max_seqs=1, **desc))
    batch = cs.cs_kv_batch(plan, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"),
                           torch.tensor([keys], dtype=torch.int32, device="cuda"),
                           torch.arange(pages, dtype=torch.int32, device="cuda")[None], tokens=tokens, max_q=tokens)
    out = torch.full((tokens, heads, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((tokens, heads), 7.0, device="cuda")
    cs.cs_kv4_attention(plan, batch, q.to(dtype).cuda(), cache(k), cache(v), out, lse)
    torch.cuda.synchronize()
    assert cs.cs_kv_status(plan) == cs.CS_OK
    return okv.to64(out), okv.to64(lse)


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("dtype,nats", [(BF16, 12), (BF16, 16), (BF16, 18), (BF16, 30), (BF16, 60), (F16, 10), (F16, 14)])
@pytest.mark.parametrize("heads,tokens,d", [(8, 1, 128), (8, 1, 64), (16, 1, 128), (4, 4, 64), (4, 40, 128)])
def test_a_key_of_nearly_all_the_weight_and_value_zero(dtype, nats, heads, tokens, d):
    """The output is that of thousands of keys whose weights are e^-nats each: as exact as these are, rounded to the dtype.

    One SM, so that a warp has many of the keys beside the one.  u |O| for the output's rounding, u sum(w |v|) for the weights', and 2^-11 sum(w |v|) for their errors from the scores (which
    are exact but for a factor in 32 bits) and the sums in 32 bits.  In f16 a tile of 128 rows rounds weights to steps of
    2^-24 of the reference, few rows 2^7 finer: half of one for each key."""
    if dtype == F16 and tokens == 40:
        nats -= 6
    g = torch.Generator().manual_seed(nats)
    keys = 4000
    q = torch.zeros(tokens, heads, d, dtype=torch.float64)
    k, v = torch.zeros(keys, 1, d, dtype=torch.float64), torch.randn(keys, 1, d, generator=g).double()
    q[..., 1], k[0, 0, 1], v[0] = 4.0, 7.0, 0.0
    scale = float(np.float32(nats / 28))
    out, lse = attend(q, k, v, dtype, scale=scale, num_sms=1)
    held_k, held_v = o4.held(k), o4.held(v)
    assert held_k[0, 0, 1] == 7.0
    u = torch.finfo(dtype).eps / 2
    for t in range(tokens):
        seen = np.arange(keys) <= keys - tokens + t
        o, z, a = okv.attend(q[t, 0], held_k[:, 0], held_v[:, 0], seen, scale)
        bound = u * np.abs(o) + (u + 2.0 ** -11) * a
        if dtype == F16:
            bound = bound + keys * 2.0 ** (-25 if tokens == 40 else -32) * np.abs(held_v).max() + 2.0 ** -25
        assert (np.abs(out[t] - o) <= bound).all(), float((np.abs(out[t] - o) / bound).max())
        assert np.abs(lse[t] - z).max() <= 2.0 ** -20 * abs(z)


# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1.0, 1e4, 1e12, 1e30])
@pytest.mark.parametrize("heads,tokens", [(8, 1), (8, 3), (8, 40)])
def test_queries_of_zeros_under_a_small_scale(dtype, size, heads, tokens):
    """Rows of zeros see all their keys alike, whatever the scale is; beside them are rows of `size`, which the scale undoes.
    Bounds: u |O|, u sum(w |v|) for the weights, 2^-11 sum(w |v|) for scores (sums of 64 products in 32 bits) and sums."""
    if dtype == F16 and size > 1e4:
        size_of_q = 1e4  # (scores of nearly 0)
    else:
        size_of_q = size
    g = torch.Generator().manual_seed(tokens)
    keys, d = 150, 64
    q = (torch.randn(tokens, heads, d, generator=g).double() * size_of_q).to(dtype).double()
    q[:, 1::2] = 0.0
    q[0, 3] = -0.0
    k, v = (torch.randn(keys, 2, d, generator=g).double() for _ in range(2))
    scale = float(np.float32(0.125 / size))
    out, lse = attend(q, k, v, dtype, scale=scale)
    held_k, held_v = o4.held(k), o4.held(v)
    u = torch.finfo(dtype).eps / 2
    for t in range(tokens):
        seen = np.arange(keys) <= keys - tokens + t
        for h in range(heads):
            o, z, a = okv.attend(q[t, h].numpy(), held_k[:, h // 4], held_v[:, h // 4], seen, scale)
            assert (np.abs(out[t, h] - o) <= u * np.abs(o) + (u + 2.0 ** -11) * a + 1e-30).all(), (t, h)
            assert abs(lse[t, h] - z) <= 2.0 ** -11 + 2.0 ** -20 * abs(z)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads,tokens", [(8, 1), (16, 1), (8, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_overflow(dtype, heads, tokens, d):
    """Scores beyond 32 bits are infinities: a key at -infinity has no weight, a row of them alone gets zeros and an lse of
    -infinity, and a row with infinity, whose softmax is no number, is NaN: as over a cache in 16 bits."""
    keys, scale = 300, 1e36
    q, k = torch.zeros(tokens, heads, d, dtype=torch.float64), torch.zeros(keys, 1, d, dtype=torch.float64)
    g = torch.Generator().manual_seed(1)
    v = torch.randn(keys, 1, d, generator=g).double()
    k[:, 0, 0] = 7.0
    k[5, 0], k[17, 0] = 0.0, 0.0
    k[5, 0, 40] = k[17, 0, 40] = 7.0
    q[..., 0] = -1e3  # -infinity but for two keys, at 0
    q[:, 1, 40] = -1e3  # everywhere
    q[:, 2, 0] = 1e3  # infinity
    out, lse = attend(q, k, v, dtype, scale=scale)
    held = o4.held(v)[:, 0]
    u = torch.finfo(dtype).eps / 2
    want = (held[5] + held[17]) / 2
    for h in [0] + list(range(3, heads)):
        assert (np.abs(out[:, h] - want) <= u * np.abs(want) + 2.0 ** -20).all()
        assert (np.abs(lse[:, h] - np.log(2)) <= 2.0 ** -20).all()
    assert (out[:, 1] == 0).all() and np.isneginf(lse[:, 1]).all()
    assert np.isnan(out[:, 2]).all() and np.isnan(lse[:, 2]).all()
    # the same through a cache in 16 bits
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=1, head_dim=d, page_size=16, num_pages=19,
                                            max_tokens=tokens, max_seqs=1, scale=scale))
    batch = cs.cs_kv_batch(plan, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), torch.tensor([keys], dtype=torch.int32,
                           device="cuda"), torch.arange(19, dtype=torch.int32, device="cuda")[None], tokens=tokens, max_q=tokens)
    kc, vc = (torch.zeros(19 * 16, 1, d, dtype=dtype, device="cuda") for _ in range(2))
    kc[:keys], vc[:keys] = torch.from_numpy(o4.held(k)).to(dtype).cuda(), torch.from_numpy(o4.held(v)).to(dtype).cuda()
    out16, lse16 = torch.empty(tokens, heads, d, dtype=dtype, device="cuda"), torch.empty(tokens, heads, device="cuda")
    cs.cs_kv_attention(plan, batch, q.to(dtype).cuda(), kc.view(19, 16, 1, d), vc.view(19, 16, 1, d), out16, lse16)
    torch.cuda.synchronize()
    out16, lse16 = okv.to64(out16), okv.to64(lse16)
    assert (np.isnan(out16) == np.isnan(out)).all() and (np.isnan(lse16) == np.isnan(lse)).all()
    assert (out16[:, 1] == 0).all() and (np.isneginf(lse16) == np.isneginf(lse)).all()


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("q,kv", [([4, 1], [70, 9]), ([6], [300]), ([200, 30], [300, 30]), ([130], [2000])])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("window,prefix", [(0, 0), (33, 0), (0, 50)])
def test_values_beyond_f16_at_keys_hidden_from_some_rows(q, kv, head_dim, window, prefix):
    """A plan of f16 over values that only a bf16 one writes, 7 times the largest scale, at keys that only the last token (or, under a
    window, only the first ones) see: every other row is as if they were not there, and rows that see one are infinite, no
    number, or right, in the group's dimensions, and right elsewhere."""
    b = Batch4(q, kv, 8, 2, head_dim, F16, window=window, sinks=2 if window else 0, prefix=prefix, seed=kv[0])
    group, spoilt = head_dim // 32 - 1, []
    dims = slice(32 * group, 32 * group + 32)
    for s, (n, m) in enumerate(zip(q, kv)):
        spoilt.append((s, m - 1))
        if window and m - n - window + 1 >= 2 and n > 1:
            spoilt.append((s, m - n - window + 1))
    for s, j in spoilt:
        page = int(b.table[s, j // 16])
        b.v4[1][page, :, j % 16, group] = 0xF7
        b.v4[0][page, j % 16, :, 16 * group:16 * group + 16] = 0xFF  # codes of 7
        b.v[s][j, :, dims] = 0.0  # rows that do not see it never read it
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
            ok = np.ones(head_dim, dtype=bool)
            ok[dims] = not hit
            assert (np.abs(got[t, :, ok] - ref[t, :, ok]) <= bound[t, :, ok]).all(), (s, i)
            t += 1


@pytest.mark.parametrize("dtype,d", [(F16, 64), (F16, 128), (BF16, 64), (BF16, 128)])
def test_no_byte_reads_back_as_what_it_does_not_stand_for(dtype, d):
    """Every scale under every code: what the dtype holds is exact, what it does not hold is infinite with its sign, and under the
    eight scales that stand for no number nothing is finite."""
    scale = np.repeat(np.arange(256), 16).reshape(-1, 1)  # [rows, 1]: each scale under 16 rotations of the codes
    code = (np.arange(d) % 16 - 8 + np.tile(np.arange(16), 256).reshape(-1, 1) + 8) % 16 - 8
    rows = len(scale)
    codes = torch.from_numpy(o4.pack(code.astype(np.int8))).view(rows // 16, 16, 1, d // 2).cuda()
    scales = torch.from_numpy(np.repeat(scale, d // 32, 1).astype(np.uint8)).view(rows // 16, 1, 16, d // 32).cuda()
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=1, kv_heads=1, head_dim=d, num_pages=rows // 16, max_tokens=rows,
                                            max_seqs=1))
    batch = cs.cs_kv_batch(plan, torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                           torch.tensor([rows], dtype=torch.int32, device="cuda"),
                           torch.arange(rows // 16, dtype=torch.int32, device="cuda")[None], tokens=rows, max_q=rows)
    k, v = (torch.empty(rows, 1, d, dtype=dtype, device="cuda") for _ in range(2))
    cs.cs_kv4_read(plan, batch, (codes, scales), (codes, scales), k, v)
    torch.cuda.synchronize()
    assert cs.cs_kv_status(plan) == cs.CS_OK
    with np.errstate(invalid="ignore"):
        want = code * o4.SCALES[scale]
    named = np.isfinite(want)
    fits = named & (np.abs(np.where(named, want, 0)) <= torch.finfo(dtype).max)
    for got in (okv.to64(k)[:, 0], okv.to64(v)[:, 0]):
        assert (got[fits] == want[fits]).all()
        assert (got[named & ~fits] == np.sign(want[named & ~fits]) * np.inf).all()
        assert not np.isfinite(got[~named]).any()
    assert (named & ~fits).any() == (dtype == F16)


def far_case(dtype, exponent, heads, tokens, d):
    """(q, k, v, scale): scores of up to 2^exponent times 40, where a step of 32 bits is many units: keys with the largest share the
    weight, the others have none of it.  Positive and negative ones, and some that rise from tile to tile."""
    keys = 400
    g = torch.Generator().manual_seed(exponent)
    q, k = torch.zeros(tokens, heads, d, dtype=torch.float64), torch.zeros(keys, 1, d, dtype=torch.float64)
    v = torch.randn(keys, 1, d, generator=g).double()
    j = torch.arange(keys)
    k[:, 0, 0] = 3.5 + 0.25 * (j % 3)
    k[:, 0, 32] = 1.0 + (j // 32) * 0.125
    q[:, 0, 0], q[:, 1, 0], q[:, 2, 32], q[:, 3, 32] = 5.3125, -5.3125, 4.6875, -4.6875
    if exponent == 0:
        q *= 8
    return q.to(dtype).double(), k, v, 2.0 ** exponent


def far_rows(q, k, v, dtype, scale):
    """(row, head, is right, lse) of each: within u |O| and u sum(w |v|) for roundings and 2^-11 sum(w |v|) for the sums; scores are
    products of one dimension each."""
    tokens, heads, _ = q.shape
    keys = len(k)
    out, lse = attend(q, k, v, dtype, scale=scale)
    held_k, held_v = o4.held(k), o4.held(v)
    u = torch.finfo(dtype).eps / 2
    for t in range(tokens):
        seen = np.arange(keys) <= keys - tokens + t
        for h in range(heads):
            o, z, a = okv.attend(q[t, h].numpy(), held_k[:, 0], held_v[:, 0], seen, scale)
            right = (np.abs(out[t, h] - o) <= u * np.abs(o) + (u + 2.0 ** -11) * a).all() and \
                abs(lse[t, h] - z) <= 2.0 ** -11 + 2.0 ** -20 * abs(z)
            yield right, np.isnan(out[t, h]).all() and np.isnan(lse[t, h]), abs(z) / math.log(2)


EXPONENTS = [0, 18, 20, 22, 24, 26, 28, 30, 40, 70, 110]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("heads,tokens,d", [(8, 1, 128), (8, 1, 64), (16, 1, 128), (4, 3, 64)])
def test_scores_far_from_zero(dtype, exponent, heads, tokens, d):
    q, k, v, scale = far_case(dtype, exponent, heads, tokens, d)
    assert all(right for right, _, _ in far_rows(q, k, v, dtype, scale))


@pytest.mark.parametrize("dtype,limit", [(F16, 2.0 ** 27), (BF16, 2.0 ** 31)])
@pytest.mark.parametrize("exponent", EXPONENTS)
@pytest.mark.parametrize("heads,tokens,d", [(4, 40, 128), (4, 150, 64), (4, 300, 128)])
def test_scores_far_from_zero_of_many_rows(dtype, limit, exponent, heads, tokens, d):
    """Beyond the limit (of base-2 scores, whose largest in a tile is within a third of the row's here) rows are NaN."""
    q, k, v, scale = far_case(dtype, exponent, heads, tokens, d)
    for right, nan, size in far_rows(q, k, v, dtype, scale):
        assert right or (nan and size >= 0.6 * limit), size
        assert nan or size <= limit, size
