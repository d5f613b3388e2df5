"""ctypes binding of the paged key/value cache held in 4 bits (``include/cs_kv4.h``).

Argument marshalling only, as in :mod:`.kv`, whose plans and batches these calls take.
A K or V cache is a pair (codes, scales) of uint8 tensors of :func:`cs_kv4_shapes`.
"""
from __future__ import annotations

import ctypes
from ctypes import byref

import torch

from .chain import Plan, _attn_args, _lib, cs_attn_args
from .kv import CS_KV_TOKEN, KVBatch, KVPlan, _bad, _check, _I, _L, _P, _rows, _same_device, _stream, _whole, cs_kv_batch_s

KV4_EXPORTED = ("cs_kv4_append", "cs_kv4_read", "cs_kv4_attention", "cs_kv4_attention_shared", "cs_attn_cached4_forward")


_K, _V = [("k_codes", _P), ("k_scales", _P)], [("v_codes", _P), ("v_scales", _P)]  # a cs_kv4_cache each


class cs_kv4_append_args(ctypes.Structure):
    _fields_ = [("qkv", _P), ("qkv_stride", _L), ("q_out", _P), ("q_stride", _L), *_K, *_V,
                ("rope", _P), ("rope_rows", _I), ("positions", _P)]


class cs_kv4_read_args(ctypes.Structure):
    _fields_ = [*_K, *_V, ("k_out", _P), ("k_stride", _L), ("v_out", _P), ("v_stride", _L)]


class cs_kv4_attn_args(ctypes.Structure):
    _fields_ = [("q", _P), ("q_stride", _L), *_K, *_V, ("out", _P), ("out_stride", _L), ("lse", _P)]


def _declare():
    B = ctypes.POINTER(cs_kv_batch_s)
    A, T = ctypes.POINTER(cs_kv4_append_args), ctypes.POINTER(cs_kv4_attn_args)
    for name, args in {
        "cs_kv4_append": [_P, B, A, _P], "cs_kv4_read": [_P, B, ctypes.POINTER(cs_kv4_read_args), _P],
        "cs_kv4_attention": [_P, B, T, _P], "cs_kv4_attention_shared": [_P, B, _P, _I, T, _P],
        "cs_attn_cached4_forward": [_P, _P, B, ctypes.POINTER(cs_attn_args), A, _P],
    }.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = _I, args


_declare()


def cs_kv4_shapes(plan: KVPlan):
    """(shape of the codes, shape of the scales) of the plan's K or V cache in 4 bits, both uint8."""
    d = plan.desc
    pages, ps, hk = d.num_pages, d.page_size, d.kv_heads
    codes = (pages, ps, hk, d.head_dim // 2) if d.cache_layout == CS_KV_TOKEN else (pages, hk, ps, d.head_dim // 2)
    return codes, (pages, hk, ps, d.head_dim // 32)


_U8 = torch.uint8


def _cache(plan, pair, name):
    """(pointer of the codes, pointer of the scales) of a cache."""
    try:
        codes_shape, scales_shape = plan._four_shapes
    except AttributeError:
        codes_shape, scales_shape = plan._four_shapes = cs_kv4_shapes(plan)
    if not isinstance(pair, (tuple, list)) or len(pair) != 2:
        raise TypeError(f"{name} must be a pair (codes, scales); got {type(pair).__name__}")
    c, s = pair
    if (isinstance(c, torch.Tensor) and isinstance(s, torch.Tensor) and c.dtype is _U8 and s.dtype is _U8
            and c.shape == codes_shape and s.shape == scales_shape and c.get_device() == s.get_device() == plan.device
            and c.is_contiguous() and s.is_contiguous()):
        return c.data_ptr(), s.data_ptr()
    _whole(c, codes_shape, _U8, plan.device, name + " codes")  # one of them says what is wrong
    _whole(s, scales_shape, _U8, plan.device, name + " scales")


def _append_args(plan, batch, k, v, rope, positions) -> cs_kv4_append_args:
    _same_device(plan, batch)
    a = cs_kv4_append_args()
    a.k_codes, a.k_scales = _cache(plan, k, "k")
    a.v_codes, a.v_scales = _cache(plan, v, "v")
    if rope is not None:
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            raise _bad("rope", rope, "a 2-D float32 tensor")
        a.rope_rows = rope.shape[0]
        a.rope = _whole(rope, (a.rope_rows, plan.desc.rotary_dim), torch.float32, plan.device, "rope")
    if positions is not None:
        a.positions = _whole(positions, (batch.tokens,), torch.int32, plan.device, "positions")
    return a


def cs_kv4_append(plan: KVPlan, batch: KVBatch, qkv, q_out, k, v, rope=None, positions=None, stream=None) -> None:
    """:func:`.kv.cs_kv_append` into the caches ``k`` and ``v`` in 4 bits."""
    a, d = _append_args(plan, batch, k, v, rope, positions), plan.desc
    a.qkv, a.qkv_stride = _rows(qkv, batch.tokens, d.heads + 2 * d.kv_heads, d.head_dim, plan.dtype, plan.device, "qkv")
    a.q_out, a.q_stride = _rows(q_out, batch.tokens, d.heads, d.head_dim, plan.dtype, plan.device, "q_out")
    if a.q_out == a.qkv and batch.tokens <= 1:
        a.q_stride = a.qkv_stride = plan.qkv_width  # one row: in place, whatever its stride
    _check(_lib.cs_kv4_append(plan.handle, batch._ref, byref(a), _stream(stream, plan.device)), "cs_kv4_append")


def cs_kv4_read(plan: KVPlan, batch: KVBatch, k, v, k_out, v_out, stream=None) -> None:
    """The values of the batch's new tokens' keys and values: ``k_out`` and ``v_out``
    [tokens, kv_heads, head_dim] of the plan's dtype.  Either may be None, and its cache then too."""
    _same_device(plan, batch)
    a, d = cs_kv4_read_args(), plan.desc
    if k_out is not None:
        a.k_codes, a.k_scales = _cache(plan, k, "k")
        a.k_out, a.k_stride = _rows(k_out, batch.tokens, d.kv_heads, d.head_dim, plan.dtype, plan.device, "k_out")
    if v_out is not None:
        a.v_codes, a.v_scales = _cache(plan, v, "v")
        a.v_out, a.v_stride = _rows(v_out, batch.tokens, d.kv_heads, d.head_dim, plan.dtype, plan.device, "v_out")
    _check(_lib.cs_kv4_read(plan.handle, batch._ref, byref(a), _stream(stream, plan.device)), "cs_kv4_read")


def _attn4_args(plan, batch, q, k, v, out, lse) -> cs_kv4_attn_args:
    _same_device(plan, batch)
    a, d = cs_kv4_attn_args(), plan.desc
    a.q, a.q_stride = _rows(q, batch.tokens, d.heads, d.head_dim, plan.dtype, plan.device, "q")
    a.out, a.out_stride = _rows(out, batch.tokens, d.heads, d.head_dim, plan.dtype, plan.device, "out")
    a.k_codes, a.k_scales = _cache(plan, k, "k")
    a.v_codes, a.v_scales = _cache(plan, v, "v")
    a.lse = None if lse is None else _whole(lse, (batch.tokens, d.heads), torch.float32, plan.device, "lse")
    return a


def cs_kv4_attention(plan: KVPlan, batch: KVBatch, q, k, v, out, lse=None, stream=None) -> None:
    """:func:`.kv.cs_kv_attention` over the caches ``k`` and ``v`` in 4 bits."""
    a = _attn4_args(plan, batch, q, k, v, out, lse)
    _check(_lib.cs_kv4_attention(plan.handle, batch._ref, byref(a), _stream(stream, plan.device)), "cs_kv4_attention")


def cs_kv4_attention_shared(plan: KVPlan, batch: KVBatch, q, k, v, prefix_pages, prefix_len: int, out, lse=None,
                            stream=None) -> None:
    """The same where every sequence's keys follow the ``prefix_len`` keys of ``prefix_pages`` (int32)."""
    a = _attn4_args(plan, batch, q, k, v, out, lse)
    if prefix_len < 0:
        raise ValueError(f"prefix_len={prefix_len}")
    need = -(-prefix_len // plan.desc.page_size)
    if not isinstance(prefix_pages, torch.Tensor) or prefix_pages.dim() != 1 or prefix_pages.shape[0] < need:
        raise _bad("prefix_pages", prefix_pages, f"a 1-D int32 tensor of at least {need} pages")
    pp = _whole(prefix_pages, tuple(prefix_pages.shape), torch.int32, plan.device, "prefix_pages")
    _check(_lib.cs_kv4_attention_shared(plan.handle, batch._ref, pp, prefix_len, byref(a), _stream(stream, plan.device)),
           "cs_kv4_attention_shared")


def cs_attn_cached4_forward(chain: Plan, plan: KVPlan, batch: KVBatch, X, Wqkv, Wo, Y, k, v, rope=None, positions=None,
                            stream=None) -> None:
    """One attention layer over caches in 4 bits: QKV = X Wqkv, append with rotation, attention, Y = O Wo."""
    args = _attn_args(chain, X, Wqkv, Wo, Y)
    for name, t in (("X", X), ("Wqkv", Wqkv), ("Wo", Wo), ("Y", Y)):
        if t is not None and t.get_device() != plan.device:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the plan on cuda:{plan.device}")
    a = _append_args(plan, batch, k, v, rope, positions)
    _check(_lib.cs_attn_cached4_forward(chain.handle, plan.handle, batch._ref, byref(args), byref(a), _stream(stream, plan.device)),
           "cs_attn_cached4_forward")
