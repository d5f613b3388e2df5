"""Which tensors the paged cache binding takes: strides of token-indexed tensors, without a
GPU.  The plan has no handle, so a call whose tensors are accepted ends in the library's
refusal of a NULL plan, before anything is read through a pointer."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

HEADS, KV_HEADS, DIM, TOKENS = 8, 2, 64, 21
WIDTH, QKV = HEADS * DIM, (HEADS + 2 * KV_HEADS) * DIM
F16 = torch.float16


@pytest.fixture(scope="module")
def cs():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import consumer_gemm_chain_gb300 as cs
    return cs


def calls(cs, tokens=TOKENS):
    """{argument: call with that argument replaced}"""
    shape = (4, 16, KV_HEADS, DIM)
    desc = cs.cs_kv_desc_init(heads=HEADS, kv_heads=KV_HEADS, head_dim=DIM)
    plan = SimpleNamespace(handle=None, device=-1, dtype=F16, desc=desc, cache_shape=shape, qkv_width=QKV,
                           _append=cs.kv.cs_kv_append_args(), _attn=cs.kv.cs_kv_attn_args())
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(tokens=tokens), (), -1)
    k, v = torch.zeros(shape, dtype=F16), torch.zeros(shape, dtype=F16)
    wide, row = torch.zeros(tokens, QKV, dtype=F16), torch.zeros(tokens, WIDTH, dtype=F16)
    pages = torch.zeros(4, dtype=torch.int32)
    return {
        "q": lambda x: cs.cs_kv_attention(plan, batch, x, k, v, row, stream=0),
        "out": lambda x: cs.cs_kv_attention(plan, batch, row, k, v, x, stream=0),
        "shared q": lambda x: cs.cs_kv_attention_shared(plan, batch, x, k, v, pages, 20, row, stream=0),
        "shared out": lambda x: cs.cs_kv_attention_shared(plan, batch, row, k, v, pages, 20, x, stream=0),
        "qkv": lambda x: cs.cs_kv_append(plan, batch, x, row, k, v, stream=0),
        "q_out": lambda x: cs.cs_kv_append(plan, batch, wide, x, k, v, stream=0),
    }


def width_of(name):
    return QKV if name == "qkv" else WIDTH


NAMES = ["q", "out", "shared q", "shared out", "qkv", "q_out"]


@pytest.mark.parametrize("name", NAMES)
def test_rows_that_share_memory_are_refused(cs, name):
    w = width_of(name)
    call = calls(cs)[name]
    one = torch.zeros(1, w, dtype=F16)
    store = torch.zeros(TOKENS * w, dtype=F16)
    for x in (one.expand(TOKENS, w), one.view(1, w // DIM, DIM).expand(TOKENS, w // DIM, DIM),
              torch.zeros((), dtype=F16), store.as_strided((TOKENS, w), (w - 8, 1)), store.as_strided((TOKENS, w // DIM, DIM), (DIM, DIM, 1))):
        with pytest.raises(ValueError, match=name.split()[-1]):
            call(x)


@pytest.mark.parametrize("name", NAMES)
def test_rows_apart_are_taken(cs, name):
    w = width_of(name)
    store = torch.zeros(TOKENS, w + 24, dtype=F16)
    for tokens, x in ((TOKENS, store[:, :w]), (TOKENS, store[:, 8:8 + w].unflatten(1, (w // DIM, DIM))),
                      (TOKENS, store[:, :w].contiguous()), (1, torch.zeros(1, w, dtype=F16)),
                      (1, torch.zeros(w, dtype=F16).expand(1, w)), (0, torch.zeros(0, w, dtype=F16))):
        with pytest.raises(cs.CSError, match="plan is NULL"):
            calls(cs, tokens)[name](x)


@pytest.mark.parametrize("length", [-1, -(1 << 32) + 100, -(1 << 31), 65, 1 << 31, (1 << 32) + 20])
def test_prefix_lengths_that_do_not_fit_the_pages(cs, length):
    """A length that 32 bits do not hold must not reach the library as another one."""
    plan = SimpleNamespace(handle=None, device=-1, dtype=F16, desc=cs.cs_kv_desc_init(heads=HEADS, kv_heads=KV_HEADS, head_dim=DIM),
                           cache_shape=(4, 16, KV_HEADS, DIM), _attn=cs.kv.cs_kv_attn_args())
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(tokens=1), (), -1)
    cache, row = torch.zeros(plan.cache_shape, dtype=F16), torch.zeros(1, WIDTH, dtype=F16)
    with pytest.raises(ValueError, match="prefix"):
        cs.cs_kv_attention_shared(plan, batch, row, cache, cache, torch.zeros(4, dtype=torch.int32), length, row, stream=0)
