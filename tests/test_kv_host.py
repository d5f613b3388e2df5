"""The paged cache operators without a GPU: exports, refusals, and the float64
definitions against independent ones."""
from __future__ import annotations

import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import kv as okv
from kv_util import Batch, rope_table

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cs():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import consumer_gemm_chain_gb300 as cs
    return cs


def test_every_declared_symbol_is_exported(cs):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "cs_kv.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(cs_[a-z0-9_]+)\s*\(", text))
    lib = ctypes.CDLL(cs.chain.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    assert names == set(cs.kv.KV_EXPORTED)
    assert cs.cs_kv_abi_version() == 1


def test_desc_defaults_and_fields(cs):
    d = cs.cs_kv_desc_init()
    assert (d.dtype, d.head_dim, d.page_size, d.cache_layout, d.window, d.scale) == (0, 128, 16, 0, 0, 0.0)
    d = cs.cs_kv_desc_init(dtype=torch.bfloat16, cache_layout="head", rotary_pairing="adjacent")
    assert (d.dtype, d.cache_layout, d.rotary_pairing) == (cs.CS_BF16, cs.CS_KV_HEAD, cs.CS_KV_ADJACENT)
    with pytest.raises(TypeError):
        cs.cs_kv_desc_init(hedas=3)


GOOD = dict(heads=8, kv_heads=2, num_pages=4, max_tokens=8, max_seqs=2)


@pytest.mark.parametrize("field,value,unsupported", [
    ("dtype", 2, 0), ("heads", 0, 0), ("heads", 2000, 0), ("kv_heads", 0, 0), ("kv_heads", 3, 0), ("head_dim", 96, 1),
    ("head_dim", 256, 1), ("page_size", 8, 1), ("page_size", 24, 1), ("page_size", 256, 1), ("num_pages", 0, 0),
    ("cache_layout", 2, 0), ("max_tokens", 0, 0), ("max_tokens", (1 << 20) + 1, 0), ("max_seqs", 0, 0), ("max_seqs", 8193, 0),
    ("rotary_dim", 8, 0), ("rotary_dim", 144, 0), ("rotary_dim", -16, 0), ("rotary_pairing", 2, 0), ("window", -1, 0),
    ("sinks", -1, 0), ("scale", -1.0, 0), ("scale", math.nan, 0), ("scale", math.inf, 0), ("shared", 2, 0), ("num_sms", -1, 0)])
def test_invalid_descs_are_rejected_without_a_gpu(cs, field, value, unsupported):
    with pytest.raises(cs.CSError) as e:
        cs.cs_kv_plan(cs.cs_kv_desc_init(**{**GOOD, field: value}))
    assert e.value.status == (cs.CS_ERR_UNSUPPORTED if unsupported else cs.CS_ERR_INVALID_ARG)


def test_combinations_that_are_refused(cs):
    for kw in (dict(shared=1, window=4), dict(heads=258, kv_heads=2)):
        with pytest.raises(cs.CSError) as e:
            cs.cs_kv_plan(cs.cs_kv_desc_init(**{**GOOD, **kw}))
        assert e.value.status == cs.CS_ERR_UNSUPPORTED


def test_null_arguments(cs):
    lib = cs.kv._lib
    assert lib.cs_kv_plan(None, None) == cs.CS_ERR_INVALID_ARG
    assert lib.cs_kv_desc_init(None) == cs.CS_ERR_INVALID_ARG
    assert lib.cs_kv_destroy(None) == cs.CS_OK
    for f in (lib.cs_kv_status, lib.cs_kv_reset):
        assert f(None) == cs.CS_ERR_INVALID_ARG
    assert lib.cs_kv_append(None, None, None, None) == cs.CS_ERR_INVALID_ARG
    assert lib.cs_kv_attention(None, None, None, None) == cs.CS_ERR_INVALID_ARG
    assert lib.cs_kv_attention_shared(None, None, None, 0, None, None) == cs.CS_ERR_INVALID_ARG
    assert lib.cs_attn_cached_forward(None, None, None, None, None, None) == cs.CS_ERR_INVALID_ARG
    assert "NULL" in cs.cs_last_error_string()


def test_the_division_of_the_work_against_counting(tmp_path):
    """The arithmetic that gives every CTA its range of key tiles, run on the host."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = tmp_path / "kv_schedule_check"
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-o", str(exe),
                    os.path.join(ROOT, "tests", "c", "kv_schedule_check.cu")], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_rotation_is_a_complex_product():
    g = np.random.default_rng(0)
    x, angle = g.standard_normal((5, 3, 16)), g.standard_normal((5, 1, 4))
    y = okv.rotate(x, np.cos(angle), np.sin(angle), "half")
    z = (x[..., :4] + 1j * x[..., 4:8]) * np.exp(1j * angle)
    assert np.allclose(y[..., :4], z.real) and np.allclose(y[..., 4:8], z.imag) and (y[..., 8:] == x[..., 8:]).all()
    y = okv.rotate(x, np.cos(angle), np.sin(angle), "adjacent")
    z = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * np.exp(1j * angle)
    assert np.allclose(y[..., 0:8:2], z.real) and np.allclose(y[..., 1:8:2], z.imag)


def test_rotated_products_depend_on_the_distance_only():
    t = okv.to64(rope_table(64, 32))
    g = np.random.default_rng(1)
    q, k = g.standard_normal(64), g.standard_normal(64)
    for pairing in ("half", "adjacent"):
        r = [[okv.rotate(q, t[a, :16], t[a, 16:], pairing) @ okv.rotate(k, t[b, :16], t[b, 16:], pairing)
              for a, b in ((5, 0), (40, 35))]]
        assert abs(r[0][0] - r[0][1]) < 1e-5  # the table holds 32-bit cosines


@pytest.mark.parametrize("window,sinks,prefix", [(0, 0, 0), (7, 0, 0), (7, 3, 0), (1, 1, 0), (0, 0, 19)])
def test_attention_definition_against_torch(window, sinks, prefix):
    b = Batch([21, 1], [30, 26], 6, 2, 64, torch.float16, window=window, sinks=sinks, prefix=prefix, poison=False)
    out, lse, _ = b.reference()
    t = 0
    for s, (n, m) in enumerate(zip(b.q_lens, b.kv_lens)):
        p = torch.arange(m - n, m)[:, None]
        j = torch.arange(m)[None]
        mask = (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p
        mask = torch.cat([torch.ones(n, prefix, dtype=torch.bool), mask], 1)
        for h in range(6):
            k, v = (torch.from_numpy(x) for x in b.keys(s, h // 3))
            q = b.q[t:t + n, h].double()
            ref = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=mask[None])[0]
            assert np.allclose(out[t:t + n, h], ref.numpy(), atol=1e-12)
            z = (q @ k.T / 8.0).masked_fill(~mask, -math.inf).logsumexp(1)
            assert np.allclose(lse[t:t + n, h], z.numpy(), atol=1e-12)
        t += n


def test_a_token_that_sees_no_key():
    b = Batch([4], [2], 2, 1, 64, torch.float16, poison=False)  # positions -2, -1, 0, 1
    out, lse, _ = b.reference()
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    assert np.allclose(out[2, 0], okv.to64(b.v[0][0, 0]))


def test_a_batch_of_another_device_is_refused(cs):
    from types import SimpleNamespace
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(), (), 1)
    plan = SimpleNamespace(device=0, _attn=None, _append=None, desc=None)
    with pytest.raises(ValueError, match="cuda:1"):
        cs.kv._kv_attn_args(plan, batch, None, None, None, None, None)
    with pytest.raises(ValueError, match="cuda:1"):
        cs.kv._append_args(plan, batch, None, None, None, None, None)
