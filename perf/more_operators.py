"""Timed cases of the paged key/value cache held in 4 bits: appending the keys and
values of new tokens (rotation, then quantising), reading them back, attention over
such a cache, and attention of a batch whose sequences share one long prefix.

A batch is as in the 16-bit cache's cases: sequence b brings q_len[b] new tokens, its
kv_len[b] keys (the new ones last) live in pages of `page_size` positions, rows behind
the last sequence are padding and are left as they were.

The format.  32 consecutive dimensions of a key (or value) of one head share a scale,
an unsigned byte of 5 exponent and 3 mantissa bits (the leading bits of a half's
magnitude): amax / 7, rounded to the nearest, at most 61440.  A value is scale * c with
c = round(x / scale) in -7 .. 7, stored as c + 8 in 4 bits; of the 8 values of a 32-bit
word, value 2 j lies at bit 4 j and value 2 j + 1 at bit 16 + 4 j.  Every scale * c is a
number of both 16-bit types.  Codes have the cache's layout, scales are always
[pages, kv_heads, page_size, head_dim / 32].
"""
import math
import random

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
_BASE = dict(dtype="bf16", heads=32, kv_heads=8, head_dim=128, page_size=16, layout="token", seqs=1, q_min=1, q_max=1,
             old_min=0, old_max=0, idle=0, pad=0, window=0, sinks=0, rotary_dim=128, pairing="half", prefix=0, lens=1)


def _case(name, op, **kw):
    c = dict(_BASE, op=op, **kw)
    c["rotary_dim"] = min(c["rotary_dim"], c["head_dim"])
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of one sequence, 12 heads of 128 as in the attention shard, written and checked: latency
        _case("append4_one_token", "append", dtype="f16", heads=12, kv_heads=12, old_min=700, old_max=700),
        # a decode step of a full serving batch, partly rotated small heads
        _case("append4_decode", "append", heads=40, kv_heads=8, head_dim=64, seqs=250, old_min=1, old_max=500, idle=3,
              rotary_dim=32, pairing="adjacent", lens=2),
        # a packed prefill of ragged prompts, its keys and values read back for the prompt's own attention
        _case("append4_prefill", "append", seqs=9, q_min=301, q_max=3001, layout="head", page_size=64, pad=5, lens=3),
        # one conversation leaves the 4-bit pool for a 16-bit one
        _case("read4_one_sequence", "read", dtype="f16", heads=12, kv_heads=12, q_min=977, q_max=977),
        # the contexts of a batch, whole, for a layer that wants them dense
        _case("read4_batch", "read", seqs=17, q_min=500, q_max=9000, page_size=32, lens=4),
        # one user's next token after a short conversation: latency
        _case("attend4_one_user", "attend", dtype="f16", heads=12, kv_heads=12, old_min=977, old_max=977),
        # a serving batch with contexts of very different lengths
        _case("attend4_long_ragged", "attend", heads=64, seqs=64, old_min=300, old_max=32000, idle=2, lens=5),
        # streaming generation with small heads: the last 1024 keys and the first 4 of long contexts
        _case("attend4_window_sinks", "attend", dtype="f16", heads=40, head_dim=64, seqs=128, old_min=500, old_max=9000,
              window=1024, sinks=4, layout="head", page_size=32, lens=6),
        # one long prompt from its first token
        _case("attend4_prompt", "attend", q_min=8192, q_max=8192, page_size=64),
        # pieces of long prompts next to single tokens of other users
        _case("attend4_pieces_mixed", "attend", heads=40, seqs=12, q_min=1, q_max=700, old_min=2000, old_max=20000, pad=7,
              layout="head", page_size=128, lens=8),
        # many samples of one long prompt, each with its own continuation
        _case("shared4_decode", "shared", seqs=128, old_min=0, old_max=600, prefix=12001, lens=9),
        # a few branches of one prompt that check a handful of proposed tokens each
        _case("shared4_branches", "shared", dtype="f16", heads=16, head_dim=64, seqs=6, q_min=1, q_max=5,
              old_min=0, old_max=150, prefix=1500, page_size=32, layout="head", lens=10),
    ]


def _seconds(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _log_int(rng, a, b):
    return max(a, min(b, round(math.exp(rng.uniform(math.log(a), math.log(b))))))


def draw(rng):
    most = max(_seconds(c) for c in listed())
    while True:
        kv_heads, group = rng.choice([(12, 1), (16, 1), (8, 4), (8, 8), (4, 7), (8, 5), (6, 3), (2, 16), (1, 12)])
        head_dim = rng.choice([64, 128, 128])
        op = rng.choice(["append", "read", "attend", "attend", "attend", "shared"])
        c = _case(None, op, dtype=rng.choice(["f16", "bf16"]), heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim,
                  page_size=rng.choice([16, 32, 64, 128]), layout=rng.choice(["token", "head"]), lens=rng.randrange(1 << 30),
                  pad=rng.choice([0, 0, 3]), rotary_dim=rng.choice([head_dim, head_dim, 32]), pairing=rng.choice(["half", "adjacent"]))
        if rng.random() < 0.5 and op != "read":  # single tokens, or a few each
            c["seqs"] = _log_int(rng, 1, 256)
            c["q_max"] = rng.choice([1, 1, 1, 4])
            c["old_max"] = _log_int(rng, 1, 32000)
            c["old_min"] = rng.randint(0, c["old_max"])
            c["idle"] = rng.choice([0, c["seqs"] // 8])
        else:  # prompts, whole or in pieces
            c["seqs"] = _log_int(rng, 1, 24)
            c["q_max"] = max(1, _log_int(rng, 24, 8192) // (c["seqs"] if op != "read" else 1))
            c["q_min"] = rng.randint(1, c["q_max"])
            c["old_max"] = rng.choice([0, _log_int(rng, 1, 8000)])
        if op == "attend" and rng.random() < 0.5:
            c["window"] = _log_int(rng, 16, 4096)
            c["sinks"] = rng.choice([0, 1, 4, 130])
        if op == "shared":
            c["prefix"] = _log_int(rng, 100, 32000)
            c["old_max"] = min(c["old_max"], 1000)
            c["old_min"] = min(c["old_min"], c["old_max"])
        if _seconds(c) <= most and _pages(c) * c["page_size"] * kv_heads * head_dim <= 2 ** 31:
            return c


def _lengths(case):
    r = random.Random(case["lens"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    kv = [n + r.randint(case["old_min"], case["old_max"]) for n in q]
    for b in r.sample(range(case["seqs"]), case["idle"]):  # a slot of the batch without a new token
        q[b] = 0
    return q, kv


def _pages(case):
    ps = case["page_size"]
    _, kv = _lengths(case)
    return sum(-(-n // ps) for n in kv) + -(-case["prefix"] // ps) + 2


def work(case):
    q, kv = _lengths(case)
    tokens, d, hq, hk = sum(q), case["head_dim"], case["heads"], case["kv_heads"]
    held = 2 * hk * (d // 2 + d // 32)  # bytes of a key and its value
    if case["op"] == "read":
        return {"bytes": tokens * (held + 4 * hk * d), "flops": tokens * 2 * hk * d}
    if case["op"] == "append":  # Q, K, V and the rotation's row in, Q and the codes out; the values read back
        return {"bytes": tokens * (2 * d * (hq + 2 * hk) + 4 * case["rotary_dim"] + 2 * d * hq + 2 * held + 4 * hk * d),
                "flops": tokens * ((hq + hk) * case["rotary_dim"] * 3 + 4 * hk * d)}
    keys = pairs = 0
    w, sinks = case["window"], case["sinks"]
    for n, m in zip(q, kv):
        if n == 0:
            continue
        first = m - n
        if w <= 0:
            keys += m
            pairs += n * first + n * (n + 1) // 2
        else:
            lo = max(0, first - w + 1)
            keys += m - lo + min(sinks, lo)
            pairs += sum(p + 1 if p < w else w + min(sinks, p - w + 1) for p in range(first, m))
    if tokens:
        keys += case["prefix"]
        pairs += tokens * case["prefix"]
    return {"bytes": keys * held + 4 * tokens * hq * d, "flops": 4 * pairs * hq * d}


def prepare(case, seed):
    dt, dev = _DT[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)
    q, kv = _lengths(case)
    d, hq, hk, ps = case["head_dim"], case["heads"], case["kv_heads"], case["page_size"]
    real = sum(q)
    tokens = real + case["pad"]
    pages = _pages(case)
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32).cpu()
    prefix_pages = -(-case["prefix"] // ps)
    cols = max(1, max(-(-n // ps) for n in kv))
    table = torch.zeros(case["seqs"], cols, dtype=torch.int32)
    at = prefix_pages
    for b, n in enumerate(kv):
        c = -(-n // ps)
        table[b, :c] = order[at:at + c]
        at += c

    def normal(*shape, size=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * size).to(dt)

    def cache():
        """Codes and scales of values near the normal distribution: scales of about 0.3."""
        shape = (pages, ps, hk, d // 8, 8) if case["layout"] == "token" else (pages, hk, ps, d // 8, 8)
        codes = torch.empty(*shape[:-1], 4, device=dev, dtype=torch.uint8)
        for i in range(0, pages, 4096):
            u = torch.randn(min(4096, pages - i), *shape[1:], generator=g, device=dev, dtype=torch.float32)
            u = u.mul_(3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
            codes[i:i + 4096] = u[..., [0, 4, 1, 5]] | u[..., [2, 6, 3, 7]] << 4
        scales = torch.randint(0x64, 0x6F, (pages, hk, ps, d // 32), generator=g, device=dev, dtype=torch.uint8)  # 0.19 to 0.47
        return codes.flatten(-2), scales

    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    s = {"case": case, "q": q, "kv": kv, "real": real, "tokens": tokens,
         "cu_q": torch.tensor(cu, dtype=torch.int32, device=dev), "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev),
         "table": table.to(dev), "prefix_table": order[:prefix_pages].to(dev), "k": cache(), "v": cache()}
    if case["op"] in ("append", "read"):
        s["k_out"], s["v_out"] = (torch.zeros(tokens, hk, d, device=dev, dtype=dt) for _ in range(2))
    if case["op"] == "append":
        s["qkv"] = normal(tokens, (hq + 2 * hk) * d)
        s["q_out"] = torch.zeros(tokens, hq, d, device=dev, dtype=dt)
        r2 = case["rotary_dim"] // 2
        angle = torch.arange(max(kv) + 1, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(r2, dtype=torch.float64) / r2)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(dev)
    elif case["op"] != "read":
        s["queries"] = normal(tokens, hq, d, size=1.5)
        s["out"] = torch.zeros(tokens, hq, d, device=dev, dtype=dt)
        # the sequences with new tokens, short contexts first
        s["order"] = sorted((b for b in range(case["seqs"]) if q[b] > 0), key=lambda b: kv[b])
        s["order_dev"] = torch.tensor(s["order"], dtype=torch.int64, device=dev)
    if own:
        import consumer_gemm_chain_gb300 as cs
        desc = cs.cs_kv_desc_init(dtype=dt, heads=hq, kv_heads=hk, head_dim=d, page_size=ps, num_pages=pages,
                                  cache_layout=case["layout"], max_tokens=max(1, tokens), max_seqs=case["seqs"],
                                  rotary_dim=case["rotary_dim"], rotary_pairing=case["pairing"], window=case["window"],
                                  sinks=case["sinks"], shared=1 if case["op"] == "shared" else 0)
        s["plan"] = cs.cs_kv_plan(desc)
        s["batch"] = cs.cs_kv_batch(s["plan"], s["cu_q"], s["kv_lens"], s["table"], tokens=tokens, max_q=max(1, max(q)))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import consumer_gemm_chain_gb300 as cs
        if op == "append":
            cs.cs_kv4_append(s["plan"], s["batch"], s["qkv"], s["q_out"], s["k"], s["v"], rope=s["rope"])
        if op in ("append", "read"):
            cs.cs_kv4_read(s["plan"], s["batch"], s["k"], s["v"], s["k_out"], s["v_out"])
        elif op == "attend":
            cs.cs_kv4_attention(s["plan"], s["batch"], s["queries"], s["k"], s["v"], s["out"])
        else:
            cs.cs_kv4_attention_shared(s["plan"], s["batch"], s["queries"], s["k"], s["v"], s["prefix_table"],
                                       s["case"]["prefix"], s["out"])
    elif op == "append":
        _append(s)
        _read(s)
    elif op == "read":
        _read(s)
    else:
        _attend(s)
    if op == "append":
        return s["q_out"], s["k_out"], s["v_out"]
    return (s["k_out"], s["v_out"]) if op == "read" else s["out"]


# ------------------------------------------------------------------ plain forms
def _place(s):
    """Sequence, position, page and slot of every new token."""
    t = torch.arange(s["real"], device="cuda")
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    pos = s["kv_lens"].long()[seq] - s["cu_q"].long()[seq + 1] + t
    ps = s["case"]["page_size"]
    return pos, s["table"].long()[seq, pos // ps], pos % ps


def _quantise(x):
    """(codes, scales) of x [..., head_dim] in 32 bits."""
    g = x.unflatten(-1, (-1, 32))
    amax = g.abs().amax(-1)
    want = amax / torch.full_like(amax, 7)  # (a plain 7 would become a product with its reciprocal)
    _, e = torch.frexp(want)
    step = torch.ldexp(torch.ones_like(want), (e - 1).clamp(min=-14) - 3)  # between neighbouring scales
    scale = ((want / step).round() * step).clamp(max=61440.0)
    c = torch.where(scale[..., None] > 0, g / scale[..., None], 0.0).round().clamp(-7, 7)
    u = (c + 8).to(torch.uint8).flatten(-2).unflatten(-1, (-1, 8))
    codes = u[..., [0, 4, 1, 5]] | u[..., [2, 6, 3, 7]] << 4
    return codes.flatten(-2), (scale.half().view(torch.int16) >> 7).to(torch.uint8)


def _values(codes, scales):
    """Values in 32 bits of codes [..., head_dim / 2] and scales [..., head_dim / 32]."""
    b = codes.unflatten(-1, (-1, 4))
    u = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return ((u.float() - 8).unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _append(s):
    c, n = s["case"], s["real"]
    d, hq, hk, rd = c["head_dim"], c["heads"], c["kv_heads"], c["rotary_dim"]
    pos, page, slot = _place(s)
    x = s["qkv"][:n].float().view(n, hq + 2 * hk, d)
    qk, v = x[:, :hq + hk], x[:, hq + hk:]
    cos, sin = s["rope"][pos][:, None, :rd // 2], s["rope"][pos][:, None, rd // 2:]
    if c["pairing"] == "half":
        a, b = qk[..., :rd // 2], qk[..., rd // 2:rd]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = qk[..., 0:rd:2], qk[..., 1:rd:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    qk = torch.cat([turned, qk[..., rd:]], -1).to(_DT[c["dtype"]])
    s["q_out"][:n] = qk[:, :hq]
    for (codes, scales), new in ((s["k"], qk[:, hq:].float()), (s["v"], v)):
        if c["layout"] == "head":
            codes = codes.transpose(1, 2)
        codes[page, slot], scales.transpose(1, 2)[page, slot] = _quantise(new)


def _read(s):
    _, page, slot = _place(s)
    for (codes, scales), out in ((s["k"], s["k_out"]), (s["v"], s["v_out"])):
        if s["case"]["layout"] == "head":
            codes = codes.transpose(1, 2)
        out[:s["real"]] = _values(codes[page, slot], scales.transpose(1, 2)[page, slot]).to(out.dtype)


def _gather(s, which, pages):
    """Values of all keys of the pages [..., n]: [..., kv_heads, n * page_size, head_dim]."""
    codes, scales = s[which]
    x = codes[pages.long()]
    if s["case"]["layout"] == "token":
        x = x.transpose(-2, -3)
    return _values(x, scales[pages.long()]).transpose(-4, -3).flatten(-3, -2)


def _attend(s):
    c = s["case"]
    d, hq, hk, ps, w, prefix = c["head_dim"], c["heads"], c["kv_heads"], c["page_size"], c["window"], c["prefix"]
    group, order = hq // hk, s["order"]
    out = torch.empty(s["tokens"] + 1, hq, d, dtype=s["out"].dtype, device="cuda")  # the last row takes what pads a chunk
    if prefix:
        before = [_gather(s, x, s["prefix_table"])[:, :prefix] for x in "kv"]
    at = 0
    while at < len(order):
        # as many sequences as fit into some GB together: their queries and keys padded to the longest
        end, n = at, 0
        while end < len(order):
            more = max(n, s["q"][order[end]])
            m = s["kv"][order[end]] + prefix
            if end > at and (end + 1 - at) * m * (hq * min(more, 1024) + 2 * hk * d) > 2 ** 28:
                break
            end, n = end + 1, more
        ids, m = s["order_dev"][at:end], s["kv"][order[end - 1]]
        pages = s["table"][ids, :-(-m // ps)]
        k, v = (_gather(s, x, pages)[:, :, :m] for x in "kv")
        if prefix:
            k, v = (torch.cat([p.expand(end - at, -1, -1, -1), x], 2) for p, x in zip(before, (k, v)))
        q0, kv = s["cu_q"].long()[ids], s["kv_lens"].long()[ids]
        count = s["cu_q"].long()[ids + 1] - q0
        j = torch.arange(-prefix, m, device="cuda")
        for i in range(0, n, 1024):
            rows = torch.arange(i, min(n, i + 1024), device="cuda")
            real = rows < count[:, None]
            where = torch.where(real, q0[:, None] + rows, s["tokens"])
            x = s["queries"][where.clamp(max=s["tokens"] - 1)].float()  # [sequences, rows, heads, d]
            x = x.unflatten(2, (hk, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
            p = ((kv - count)[:, None] + rows)[..., None]
            hidden = j > p
            if w > 0:
                hidden = hidden | ((j <= p - w) & (j >= c["sinks"]))
            z = (x @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).unflatten(2, (group, -1))
            z = z.masked_fill_(hidden[:, None, None], -math.inf).flatten(2, 3)
            z = z.sub_(z.amax(-1, keepdim=True)).exp_()
            y = (z @ v) / z.sum(-1, keepdim=True)
            out[where] = y.unflatten(2, (group, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3).to(out.dtype)
        at = end
    s["out"][:s["real"]] = out[:s["real"]]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_read(s) if case["op"] == "read" else _exact_attend(s)


def _scale_of_byte():
    """The 256 scales in 64 bits (the last 8 stand for no number)."""
    b = torch.arange(256, device="cuda")
    e, f = b // 8, (b % 8).double()
    x = torch.where(e == 0, f / 8, 1 + f / 8) * 2.0 ** (e.clamp(min=1) - 15).double()
    return torch.where(b >= 0xF8, math.nan, x)


_WORD = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of a word at which its value 0, 1, ... lies, counted in bits of 4


def _keys(s, which, page, slot, h):
    """Values in 64 bits at pages and slots [n] of head h: [n, head_dim]."""
    codes, scales = s[which]
    x = codes[page, slot, h] if s["case"]["layout"] == "token" else codes[page, h, slot]
    words = x.contiguous().view(torch.int32)
    nibbles = torch.stack([words >> 4 * i & 15 for i in _WORD], -1).double() - 8.0
    return nibbles.flatten(1) * _scale_of_byte()[scales[page, h, slot].long()].repeat_interleave(32, 1)


def _exact_read(s):
    ps, hk, outs = s["case"]["page_size"], s["case"]["kv_heads"], []
    table = s["table"].long()
    for which in "kv":
        out = s[which + "_out"].double()
        at = 0
        for b, (n, m) in enumerate(zip(s["q"], s["kv"])):
            p = torch.arange(m - n, m, device="cuda")
            for h in range(hk):
                out[at:at + n, h] = _keys(s, which, table[b, p // ps], p % ps, h)
            at += n
        outs.append(out)
    return tuple(outs)


def _exact_append(s):
    c = s["case"]
    d, hq, hk, half = c["head_dim"], c["heads"], c["kv_heads"], c["rotary_dim"] // 2
    q_out, k_out, v_out = s["q_out"].double(), s["k_out"].double(), s["v_out"].double()
    scales = _scale_of_byte()[:0xF8]

    def held(x):
        """What 4 bits and a scale make of x [tokens, heads, head_dim]."""
        y = x.reshape(*x.shape[:2], d // 32, 32)
        amax = y.abs().max(-1).values
        at = torch.searchsorted(7 * scales, amax).clamp(1, len(scales) - 1)  # the scales below and above
        lo, hi = scales[at - 1], scales[at]
        up = (amax - 7 * lo > 7 * hi - amax) | ((amax - 7 * lo == 7 * hi - amax) & (at % 2 == 0))
        f = torch.where(up, hi, lo)[..., None]
        return torch.where(f == 0, torch.zeros_like(y), torch.round(y / f).clamp(-7, 7) * f).reshape(x.shape)

    at = 0
    for n, m in zip(s["q"], s["kv"]):
        if n == 0:
            continue
        rows = s["qkv"][at:at + n].double().reshape(n, hq + 2 * hk, d)
        turn = torch.complex(s["rope"][m - n:m, :half].double(), s["rope"][m - n:m, half:].double())[:, None]
        qk = rows[:, :hq + hk].clone()
        i = torch.arange(half, device="cuda")
        lo, hi = (i, i + half) if c["pairing"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(qk[..., lo], qk[..., hi]) * turn
        qk[..., lo], qk[..., hi] = z.real, z.imag
        q_out[at:at + n] = qk[:, :hq]
        k_out[at:at + n] = held(qk[:, hq:].to(s["qkv"].dtype).double())  # a key is rounded to its type, then held
        v_out[at:at + n] = held(rows[:, hq + hk:])
        at += n
    return q_out, k_out, v_out


def _exact_attend(s):
    c = s["case"]
    if work(c)["flops"] > 6e12:
        return None
    d, hk, ps, group, prefix = c["head_dim"], c["kv_heads"], c["page_size"], c["heads"] // c["kv_heads"], c["prefix"]
    out, at = s["out"].double(), 0
    first = torch.arange(prefix, device="cuda")
    for b, (n, m) in enumerate(zip(s["q"], s["kv"])):
        if n == 0:
            continue
        own_keys = torch.arange(m, device="cuda")
        page = torch.cat([s["prefix_table"].long()[first // ps], s["table"][b].long()[own_keys // ps]])
        slot = torch.cat([first % ps, own_keys % ps])
        place = torch.arange(len(page), device="cuda")
        for h in range(hk):
            k, v = (_keys(s, x, page, slot, h) for x in "kv")
            for i in range(0, n, 256):
                e = min(n, i + 256)
                x = s["queries"][at + i:at + e, h * group:(h + 1) * group].double()
                score = torch.einsum("tgd,kd->tgk", x, k) / d ** 0.5
                back = (torch.arange(i, e, device="cuda") + len(page) - n)[:, None] - place[None]  # how far the key lies behind
                seen = back >= 0
                if c["window"] > 0:
                    seen &= (back < c["window"]) | (place < c["sinks"])[None]
                score = torch.where(seen[:, None], score, float("-inf"))
                weight = torch.exp(score - torch.logsumexp(score, -1, keepdim=True))
                out[at + i:at + e, h * group:(h + 1) * group] = torch.einsum("tgk,kd->tgd", weight, v)
        at += n
    return out
