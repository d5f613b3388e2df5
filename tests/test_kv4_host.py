"""The paged cache in 4 bits without a GPU: exports, refusals, the binding, and the format's
definition against independent ones."""
from __future__ import annotations

import ctypes
import os
import re
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv_programs
from kv4_util import parts
from oracle import kv4 as o4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADS, KV_HEADS, DIM, TOKENS, PAGES = 8, 2, 64, 21, 4
WIDTH, QKV, KV = HEADS * DIM, (HEADS + 2 * KV_HEADS) * DIM, KV_HEADS * DIM
F16 = torch.float16


@pytest.fixture(scope="module")
def cs():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import consumer_gemm_chain_gb300 as cs
    return cs


def test_every_declared_symbol_is_exported(cs):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cs_kv4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(cs_[a-z0-9_]+)\s*\(", text))
    lib = ctypes.CDLL(cs.chain.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    assert names == set(cs.kv4.KV4_EXPORTED)


def test_what_is_refused_on_the_host(tmp_path):
    assert kv_programs.run("kv4_host_check", tmp_path) == (0, "ok")


# ------------------------------------------------------------------ the format
def test_a_scale_is_the_half_of_its_byte():
    half = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(half[:0xF8], o4.SCALES[:0xF8]) and not np.isfinite(half[0xF8:]).any()
    assert o4.SCALES[0xF7] == 61440 and o4.SCALES[1] == 2.0 ** -17


def test_held_values_are_numbers_of_both_types():
    v = o4.SCALES[:0xF8, None] * np.arange(-8, 8)
    for dtype in (torch.float16, torch.bfloat16):
        t = torch.from_numpy(v).to(dtype).double().numpy()
        fits = np.abs(v) <= torch.finfo(dtype).max
        assert np.array_equal(t[fits], v[fits])


def test_quantising_against_search():
    """No other scale is nearer to max / 7 and no other code nearer to x; ties go to even."""
    g = np.random.default_rng(0)
    x = g.standard_normal((400, 32)) * 2.0 ** g.integers(-24, 18, (400, 1))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    c, byte = o4.quantise(x)
    for row, codes, b in zip(x, c, byte[:, 0]):
        want = np.abs(row).max() / 7
        far = np.abs(o4.FINITE - want)
        assert far[b] == far.min()
        for e, code in zip(row, codes):
            d = np.abs(o4.SCALES[b] * np.arange(-7, 8) - e)
            assert d[code + 7] == d.min()
    s = o4.SCALES[0x70]
    c, byte = o4.quantise(np.array([7 * s, 0.5 * s, 1.5 * s, 2.5 * s, -0.5 * s, -3.5 * s] + [0.0] * 26))
    assert byte[0] == 0x70 and c[:6].tolist() == [7, 0, 2, 2, 0, -4]
    for b in (0x70, 0x71):  # the middle between two scales: the even byte
        assert o4.quantise(np.full(32, 7 * (o4.SCALES[b] + o4.SCALES[b + 1]) / 2))[1][0] == b + (b & 1)


def test_rounding_by_sums():
    """The kernel's quotients, in the same steps: x times the rounded reciprocal plus 192 (one rounding), plus 1.5 2^23 + 8 - 192.
    Every scale against every value of both types that it can meet."""
    f = np.float32
    values = {16: np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64),
              8: (np.arange(0x7F80, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)}
    for byte in range(1, 0xF8):
        s = o4.SCALES[byte]
        for x in values.values():
            x = x[x <= 60 * s]
            x = np.concatenate([x, -x])
            inv = np.float64(f(1) / f(s))
            r = (x * inv + 192.0).astype(f) + f(12582728)  # (the product and sum fit 53 bits)
            code = np.clip(r, f(12582913), f(12582927)).view(np.uint32) & 15
            assert np.array_equal(code, np.clip(np.rint(x / s), -7, 7) + 8)


def test_the_stated_error():
    g = np.random.default_rng(1)
    x = g.standard_normal((2000, 32)) * 2.0 ** g.uniform(-11, 15, (2000, 1))
    top = np.abs(x).max(-1)
    x = x[(top / 7 >= 2.0 ** -14) & (top / 7 <= 61440)]
    c, byte = o4.quantise(x)
    s = o4.SCALES[byte]
    assert (np.abs(x - o4.values(c, byte)) <= 0.54 * s).all()
    assert np.abs(o4.held(np.full(32, 1e9))).max() == 430080


def test_zeros_and_values_that_are_not_finite():
    x = np.zeros((2, 64))
    x[1, 40] = np.nan
    c, byte = o4.quantise(x)
    assert (c == 0).all() and byte.tolist() == [[0, 0], [0, 0xFF]]
    assert np.isnan(o4.values(c, byte)[1, 32:]).all() and (o4.values(c, byte)[0] == 0).all()


def test_packing():
    c = np.arange(-7, 9 - 8).repeat(1)[:8]
    word = int(o4.pack(c).view("<u4")[0])
    for v in range(8):
        assert word >> (4 * (v // 2) + 16 * (v % 2)) & 15 == c[v] + 8
    g = np.random.default_rng(2).integers(-8, 8, (3, 5, 128))
    assert np.array_equal(o4.unpack(o4.pack(g)), g)


def test_plain_form_of_the_timed_cases_agrees():
    from perf import more_operators as m
    g = torch.Generator().manual_seed(0)
    t = torch.randn(300, 128, generator=g) * torch.exp2(torch.randint(-26, 12, (300, 1), generator=g).float())
    t = t.to(torch.bfloat16).float()
    t[0] = 0
    codes, scales = m._quantise(t)
    c, byte = o4.quantise(t)
    assert np.array_equal(codes.numpy(), o4.pack(c)) and np.array_equal(scales.numpy(), byte)
    assert np.array_equal(m._values(codes, scales).double().numpy(), o4.held(t))


def test_layouts():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 16, 2, 64, generator=g)
    a, b = parts(x, "token"), parts(x.transpose(1, 2).contiguous(), "head")
    assert a[0].shape == (3, 16, 2, 32) and torch.equal(a[0].transpose(1, 2), b[0])
    assert a[1].shape == (3, 2, 16, 2) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ the binding
def calls(cs, tokens=TOKENS):
    """{argument: call with that argument replaced}; the plan has no handle, so a call whose tensors are taken ends in
    the library's refusal of a NULL plan."""
    desc = cs.cs_kv_desc_init(heads=HEADS, kv_heads=KV_HEADS, head_dim=DIM, num_pages=PAGES)
    plan = SimpleNamespace(handle=None, device=-1, dtype=F16, desc=desc, qkv_width=QKV)
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(tokens=tokens), (), -1)
    codes, scales = cs.cs_kv4_shapes(plan)
    k, v = ((torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8)) for _ in range(2))
    wide, row, held = (torch.zeros(tokens, w, dtype=F16) for w in (QKV, WIDTH, KV))
    pages = torch.zeros(4, dtype=torch.int32)
    return {
        "q": lambda x: cs.cs_kv4_attention(plan, batch, x, k, v, row, stream=0),
        "out": lambda x: cs.cs_kv4_attention(plan, batch, row, k, v, x, stream=0),
        "shared q": lambda x: cs.cs_kv4_attention_shared(plan, batch, x, k, v, pages, 20, row, stream=0),
        "shared out": lambda x: cs.cs_kv4_attention_shared(plan, batch, row, k, v, pages, 20, x, stream=0),
        "qkv": lambda x: cs.cs_kv4_append(plan, batch, x, row, k, v, stream=0),
        "q_out": lambda x: cs.cs_kv4_append(plan, batch, wide, x, k, v, stream=0),
        "k_out": lambda x: cs.cs_kv4_read(plan, batch, k, v, x, held, stream=0),
        "v_out": lambda x: cs.cs_kv4_read(plan, batch, k, v, held, x, stream=0),
    }, {
        "attention": lambda c: cs.cs_kv4_attention(plan, batch, row, c, v, torch.zeros_like(row), stream=0),
        "shared": lambda c: cs.cs_kv4_attention_shared(plan, batch, row, k, c, pages, 20, torch.zeros_like(row), stream=0),
        "append": lambda c: cs.cs_kv4_append(plan, batch, wide, row, k, c, stream=0),
        "read": lambda c: cs.cs_kv4_read(plan, batch, c, v, held, None, stream=0),
    }, k


NAMES = ["q", "out", "shared q", "shared out", "qkv", "q_out", "k_out", "v_out"]


def width_of(name):
    return QKV if name == "qkv" else KV if name in ("k_out", "v_out") else WIDTH


@pytest.mark.parametrize("name", NAMES)
def test_rows_that_share_memory_are_refused(cs, name):
    w = width_of(name)
    call = calls(cs)[0][name]
    one = torch.zeros(1, w, dtype=F16)
    store = torch.zeros(TOKENS * w, dtype=F16)
    for x in (one.expand(TOKENS, w), torch.zeros((), dtype=F16), store.as_strided((TOKENS, w), (w - 8, 1)),
              torch.zeros(TOKENS, w), torch.zeros(TOKENS + 1, w, dtype=F16), torch.zeros(w, TOKENS, dtype=F16).t()):
        with pytest.raises(ValueError, match=name.split()[-1]):
            call(x)


@pytest.mark.parametrize("name", NAMES)
def test_rows_apart_are_taken(cs, name):
    w = width_of(name)
    store = torch.zeros(TOKENS, w + 24, dtype=F16)
    for tokens, x in ((TOKENS, store[:, :w]), (TOKENS, store[:, 8:8 + w].unflatten(1, (w // DIM, DIM))), (1, torch.zeros(1, w, dtype=F16)),
                      (0, torch.zeros(0, w, dtype=F16))):
        with pytest.raises(cs.CSError, match="plan is NULL"):
            calls(cs, tokens)[0][name](x)


@pytest.mark.parametrize("name", ["attention", "shared", "append", "read"])
def test_caches(cs, name):
    _, by_cache, k = calls(cs)
    call = by_cache[name]
    with pytest.raises(cs.CSError, match="plan is NULL"):
        call((k[0].clone(), k[1].clone()))
    with pytest.raises(cs.CSError, match="plan is NULL"):
        call([k[0].clone(), k[1].clone()])
    for bad in (k[0], None, (k[0],), (k[0], k[1], k[1])):
        with pytest.raises(TypeError, match="codes, scales"):
            call(bad)
    for bad in ((k[1], k[0]), (k[0].to(torch.int8), k[1]), (k[0], k[1].float()), (k[0][:2], k[1]), (k[0], k[1][..., :1]),
                (torch.zeros(PAGES, KV_HEADS, 16, DIM // 2, dtype=torch.uint8).transpose(1, 2), k[1])):
        with pytest.raises(ValueError, match="codes|scales"):
            call(bad)


def test_another_device_and_bad_prefixes(cs):
    desc = cs.cs_kv_desc_init(heads=HEADS, kv_heads=KV_HEADS, head_dim=DIM, num_pages=PAGES)
    plan = SimpleNamespace(handle=None, device=0, dtype=F16, desc=desc)
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(), (), 1)
    for call in (lambda: cs.cs_kv4_attention(plan, batch, None, None, None, None), lambda: cs.cs_kv4_read(plan, batch, None, None, None, None),
                 lambda: cs.cs_kv4_append(plan, batch, None, None, None, None)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    plan = SimpleNamespace(handle=None, device=-1, dtype=F16, desc=desc)
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(tokens=1), (), -1)
    codes, scales = cs.cs_kv4_shapes(plan)
    pair = torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8)
    row = torch.zeros(1, WIDTH, dtype=F16)
    for length in (-1, -(1 << 32) + 100, 65, 1 << 31, (1 << 32) + 20):
        with pytest.raises(ValueError, match="prefix"):
            cs.cs_kv4_attention_shared(plan, batch, row, pair, pair, torch.zeros(4, dtype=torch.int32), length, row, stream=0)
    for pages in (None, torch.zeros(4), torch.zeros(2, 2, dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError), match="prefix_pages"):
            cs.cs_kv4_attention_shared(plan, batch, row, pair, pair, pages, 20, row, stream=0)


def test_long_items_of_few_rows_are_cut(tmp_path):
    assert kv_programs.run("kv4_uncut_check", tmp_path) == (0, "ok")
