"""ctypes binding of the paged key/value cache operators (``include/cs_kv.h``).

Argument marshalling only, as in :mod:`.chain`: tensors become device pointers,
the current torch stream becomes a ``cudaStream_t``.
"""
from __future__ import annotations

import ctypes
from ctypes import byref

import torch

from .chain import CS_BF16, CS_OK, CSError, _dtype_code, _lib, _stream_ptr
from .chain import Plan, _attn_args, cs_attn_args

CS_KV_TOKEN, CS_KV_HEAD = 0, 1
CS_KV_HALF, CS_KV_ADJACENT = 0, 1
KV_LAYOUTS = {"token": CS_KV_TOKEN, "head": CS_KV_HEAD}
KV_PAIRINGS = {"half": CS_KV_HALF, "adjacent": CS_KV_ADJACENT}

KV_EXPORTED = ("cs_kv_desc_init", "cs_kv_plan", "cs_kv_destroy", "cs_kv_append", "cs_kv_attention",
               "cs_kv_attention_shared", "cs_attn_cached_forward", "cs_kv_status", "cs_kv_reset", "cs_kv_abi_version")

_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong


class cs_kv_desc(ctypes.Structure):
    _fields_ = [("dtype", _I), ("heads", _I), ("kv_heads", _I), ("head_dim", _I), ("page_size", _I), ("num_pages", _I),
                ("cache_layout", _I), ("max_tokens", _I), ("max_seqs", _I), ("rotary_dim", _I), ("rotary_pairing", _I),
                ("window", _I), ("sinks", _I), ("scale", ctypes.c_float), ("shared", _I), ("num_sms", _I)]


class cs_kv_batch_s(ctypes.Structure):
    _fields_ = [("tokens", _I), ("seqs", _I), ("max_q", _I), ("table_cols", _I), ("cu_q", _P), ("kv_lens", _P),
                ("page_table", _P)]


class cs_kv_append_args(ctypes.Structure):
    _fields_ = [("qkv", _P), ("qkv_stride", _L), ("q_out", _P), ("q_stride", _L), ("k_cache", _P), ("v_cache", _P),
                ("rope", _P), ("rope_rows", _I), ("positions", _P)]


class cs_kv_attn_args(ctypes.Structure):
    _fields_ = [("q", _P), ("q_stride", _L), ("k_cache", _P), ("v_cache", _P), ("out", _P), ("out_stride", _L),
                ("lse", _P)]


def _declare():
    D, B = ctypes.POINTER(cs_kv_desc), ctypes.POINTER(cs_kv_batch_s)
    A, T = ctypes.POINTER(cs_kv_append_args), ctypes.POINTER(cs_kv_attn_args)
    for name, args in {
        "cs_kv_desc_init": [D], "cs_kv_plan": [D, ctypes.POINTER(_P)], "cs_kv_destroy": [_P],
        "cs_kv_append": [_P, B, A, _P], "cs_kv_attention": [_P, B, T, _P],
        "cs_kv_attention_shared": [_P, B, _P, _I, T, _P],
        "cs_attn_cached_forward": [_P, _P, B, ctypes.POINTER(cs_attn_args), A, _P],
        "cs_kv_status": [_P], "cs_kv_reset": [_P], "cs_kv_abi_version": [],
    }.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = _I, args


_declare()


# torch's current stream as an integer (what torch.cuda.current_stream().cuda_stream
# gives, without the stream object: 0.1 us against 3.2 us on a Grace core)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream_ptr(stream)


def _check(status: int, what: str) -> None:
    if status != CS_OK:
        raise CSError(status, what)


def cs_kv_abi_version() -> int:
    return _lib.cs_kv_abi_version()


def cs_kv_desc_init(**fields) -> cs_kv_desc:
    """A desc with the library defaults, then ``fields`` applied (names as in the C
    struct; ``dtype`` accepts torch dtypes, ``cache_layout`` "token"/"head",
    ``rotary_pairing`` "half"/"adjacent")."""
    d = cs_kv_desc()
    _check(_lib.cs_kv_desc_init(byref(d)), "cs_kv_desc_init")
    names = {n for n, _ in cs_kv_desc._fields_}
    for k, v in fields.items():
        if k not in names:
            raise TypeError(f"cs_kv_desc has no field {k!r}")
        if k == "dtype" and not isinstance(v, int):
            v = _dtype_code(v)
        elif k == "cache_layout" and isinstance(v, str):
            v = KV_LAYOUTS[v]
        elif k == "rotary_pairing" and isinstance(v, str):
            v = KV_PAIRINGS[v]
        setattr(d, k, v)
    return d


class KVPlan:
    """Handle of a plan made by :func:`cs_kv_plan` (destroy with :func:`cs_kv_destroy`)."""

    def __init__(self, handle: int, desc: cs_kv_desc, device: int):
        self.handle = handle
        self.desc = desc
        self.device = device
        self.dtype = torch.bfloat16 if desc.dtype == CS_BF16 else torch.float16
        d, ps, hk = desc.head_dim, desc.page_size, desc.kv_heads
        self.cache_shape = (desc.num_pages, ps, hk, d) if desc.cache_layout == CS_KV_TOKEN else (desc.num_pages, hk, ps, d)
        self.q_width = desc.heads * d
        self.qkv_width = (desc.heads + 2 * hk) * d
        # argument blocks filled by every call (a plan belongs to one thread at a time)
        self._append, self._attn = cs_kv_append_args(), cs_kv_attn_args()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        cs_kv_destroy(self)

    def __del__(self):
        try:
            cs_kv_destroy(self)
        except Exception:
            pass


def cs_kv_plan(desc: cs_kv_desc) -> KVPlan:
    h = _P()
    _check(_lib.cs_kv_plan(byref(desc), byref(h)), "cs_kv_plan")
    d = cs_kv_desc()
    ctypes.memmove(byref(d), byref(desc), ctypes.sizeof(desc))
    return KVPlan(h.value, d, torch.cuda.current_device())


def cs_kv_destroy(plan: KVPlan) -> None:
    if plan is not None and plan.handle:
        h, plan.handle = plan.handle, None
        _check(_lib.cs_kv_destroy(h), "cs_kv_destroy")


def _bad(name, t, want):
    got = f"{type(t).__name__}" if not isinstance(t, torch.Tensor) else \
        f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}"
    kind = TypeError if not isinstance(t, torch.Tensor) else ValueError
    return kind(f"{name} must be {want}; got {got}")


def _whole(t, shape, dtype, device, name) -> int:
    """Pointer of a contiguous tensor of this shape, dtype and device."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or t.get_device() != device
            or not t.is_contiguous()):
        raise _bad(name, t, f"a contiguous {shape} {dtype} tensor on cuda:{device}")
    return t.data_ptr()


def _rows(t, tokens, heads, head_dim, dtype, device, name):
    """(pointer, row stride) of a token-indexed tensor: [tokens, width] or
    [tokens, heads, head_dim], each row contiguous, rows at least their width apart
    (a broadcast row's stride 0 would mean "packed rows" to the library)."""
    width = heads * head_dim
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device:
        shape, stride = t.shape, t.stride()
        if ((len(shape) == 2 and shape[0] == tokens and shape[1] == width and stride[1] == 1) or (
                len(shape) == 3 and shape[0] == tokens and shape[1] == heads and shape[2] == head_dim
                and stride[2] == 1 and (stride[1] == head_dim or heads == 1))) and (tokens <= 1 or stride[0] >= width):
            return t.data_ptr(), stride[0] if tokens > 1 else 0
    raise _bad(name, t, f"a [{tokens}, {width}] or [{tokens}, {heads}, {head_dim}] {dtype} tensor on "
                        f"cuda:{device} with contiguous rows that do not overlap")


class KVBatch:
    """One batch (see ``cs_kv_batch`` in include/cs_kv.h); keeps its tensors alive."""

    def __init__(self, raw: cs_kv_batch_s, tensors, device: int):
        self.raw = raw
        self.device = device
        self.tokens = raw.tokens
        self.tensors = tensors
        self._ref = byref(raw)


def cs_kv_batch(plan: KVPlan, cu_q, kv_lens, page_table, tokens: int, max_q: int) -> KVBatch:
    """The batch of a step, for every call of that step (all layers): ``cu_q`` [seqs + 1],
    ``kv_lens`` [seqs] and ``page_table`` [seqs, cols], int32 on the plan's device.
    Their contents are read when the calls run."""
    if not isinstance(kv_lens, torch.Tensor) or kv_lens.dim() != 1:
        raise _bad("kv_lens", kv_lens, "a 1-D int32 tensor")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise _bad("page_table", page_table, "a 2-D int32 tensor")
    seqs, cols = kv_lens.shape[0], page_table.shape[1]
    b = cs_kv_batch_s(tokens=tokens, seqs=seqs, max_q=max_q, table_cols=cols)
    b.cu_q = _whole(cu_q, (seqs + 1,), torch.int32, plan.device, "cu_q")
    b.kv_lens = _whole(kv_lens, (seqs,), torch.int32, plan.device, "kv_lens")
    b.page_table = _whole(page_table, (seqs, cols), torch.int32, plan.device, "page_table")
    return KVBatch(b, (cu_q, kv_lens, page_table), plan.device)


def _same_device(plan, batch) -> None:
    if batch.device != plan.device:
        raise ValueError(f"the batch is on cuda:{batch.device}, the plan on cuda:{plan.device}")


def _append_args(plan, batch, a, k_cache, v_cache, rope, positions):
    _same_device(plan, batch)
    a.k_cache = _whole(k_cache, plan.cache_shape, plan.dtype, plan.device, "k_cache")
    a.v_cache = _whole(v_cache, plan.cache_shape, plan.dtype, plan.device, "v_cache")
    if rope is None:
        a.rope, a.rope_rows = None, 0
    else:
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            raise _bad("rope", rope, "a 2-D float32 tensor")
        a.rope_rows = rope.shape[0]
        a.rope = _whole(rope, (a.rope_rows, plan.desc.rotary_dim), torch.float32, plan.device, "rope")
    a.positions = None if positions is None else _whole(positions, (batch.tokens,), torch.int32, plan.device, "positions")


def cs_kv_append(plan: KVPlan, batch: KVBatch, qkv, q_out, k_cache, v_cache, rope=None, positions=None, stream=None) -> None:
    """Rotate Q and K of ``qkv`` ([tokens, (heads + 2 kv_heads) * head_dim]) by the angles of
    ``rope`` ([rows, rotary_dim]: cosines, then sines), write Q to ``q_out`` (which may be
    ``qkv[:, :heads * head_dim]`` itself) and K, V to the cache."""
    a, d = plan._append, plan.desc
    a.qkv, a.qkv_stride = _rows(qkv, batch.tokens, d.heads + 2 * d.kv_heads, d.head_dim, plan.dtype, plan.device, "qkv")
    a.q_out, a.q_stride = _rows(q_out, batch.tokens, d.heads, d.head_dim, plan.dtype, plan.device, "q_out")
    if a.q_out == a.qkv and batch.tokens <= 1:
        a.q_stride = a.qkv_stride = plan.qkv_width  # one row: in place, whatever its stride
    _append_args(plan, batch, a, k_cache, v_cache, rope, positions)
    _check(_lib.cs_kv_append(plan.handle, batch._ref, byref(a), _stream(stream, plan.device)), "cs_kv_append")


def _kv_attn_args(plan, batch, q, k_cache, v_cache, out, lse):
    _same_device(plan, batch)
    a, d = plan._attn, plan.desc
    a.q, a.q_stride = _rows(q, batch.tokens, d.heads, d.head_dim, plan.dtype, plan.device, "q")
    a.out, a.out_stride = _rows(out, batch.tokens, d.heads, d.head_dim, plan.dtype, plan.device, "out")
    a.k_cache = _whole(k_cache, plan.cache_shape, plan.dtype, plan.device, "k_cache")
    a.v_cache = _whole(v_cache, plan.cache_shape, plan.dtype, plan.device, "v_cache")
    a.lse = None if lse is None else _whole(lse, (batch.tokens, d.heads), torch.float32, plan.device, "lse")
    return a


def cs_kv_attention(plan: KVPlan, batch: KVBatch, q, k_cache, v_cache, out, lse=None, stream=None) -> None:
    """Attention of the batch's new tokens over the cache: ``q`` and ``out`` [tokens, heads, head_dim],
    ``lse`` (optional) float32 [tokens, heads]."""
    a = _kv_attn_args(plan, batch, q, k_cache, v_cache, out, lse)
    _check(_lib.cs_kv_attention(plan.handle, batch._ref, byref(a), _stream(stream, plan.device)), "cs_kv_attention")


def cs_kv_attention_shared(plan: KVPlan, batch: KVBatch, q, k_cache, v_cache, prefix_pages, prefix_len: int, out, lse=None,
                           stream=None) -> None:
    """The same where every sequence's keys follow the ``prefix_len`` keys of ``prefix_pages`` (int32)."""
    a = _kv_attn_args(plan, batch, q, k_cache, v_cache, out, lse)
    if prefix_len < 0:
        raise ValueError(f"prefix_len={prefix_len}")
    need = -(-prefix_len // plan.desc.page_size)
    if not isinstance(prefix_pages, torch.Tensor) or prefix_pages.dim() != 1 or prefix_pages.shape[0] < need:
        raise _bad("prefix_pages", prefix_pages, f"a 1-D int32 tensor of at least {need} pages")
    pp = _whole(prefix_pages, tuple(prefix_pages.shape), torch.int32, plan.device, "prefix_pages")
    _check(_lib.cs_kv_attention_shared(plan.handle, batch._ref, pp, prefix_len, byref(a), _stream(stream, plan.device)),
           "cs_kv_attention_shared")


def cs_attn_cached_forward(chain: Plan, plan: KVPlan, batch: KVBatch, X, Wqkv, Wo, Y, k_cache, v_cache, rope=None,
                           positions=None, stream=None) -> None:
    """One attention layer over the cache: QKV = X Wqkv, append with rotation, attention, Y = O Wo."""
    args = _attn_args(chain, X, Wqkv, Wo, Y)
    for name, t in (("X", X), ("Wqkv", Wqkv), ("Wo", Wo), ("Y", Y)):
        if t is not None and t.get_device() != plan.device:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the plan on cuda:{plan.device}")
    a = plan._append
    _append_args(plan, batch, a, k_cache, v_cache, rope, positions)
    _check(_lib.cs_attn_cached_forward(chain.handle, plan.handle, batch._ref, byref(args), byref(a), _stream(stream, plan.device)),
           "cs_attn_cached_forward")


def cs_kv_status(plan: KVPlan) -> int:
    """Device status of the plan's calls so far (after a stream sync): a cs_status code."""
    return _lib.cs_kv_status(plan.handle)


def cs_kv_reset(plan: KVPlan) -> None:
    _check(_lib.cs_kv_reset(plan.handle), "cs_kv_reset")
