"""Timed cases of the paged key/value cache operators: appending the keys and
values of new tokens (with the rotation of queries and keys), attention over the
cache, and attention of a batch whose sequences share one long prefix.

A batch holds `seqs` sequences.  Sequence b brings q_len[b] new tokens; its keys
0 .. kv_len[b]-1 (the new ones last) live in pages of `page_size` positions, which
its row of the page table names.  New tokens of all sequences lie one after
another in the token-indexed tensors; rows behind the last sequence are padding
and are left as they were.
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
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of one sequence, 12 heads of 128 as in the attention shard: pure latency
        _case("append_one_token", "append", dtype="f16", heads=12, kv_heads=12, old_min=700, old_max=700),
        # a decode step of a full serving batch
        _case("append_decode_256", "append", heads=64, seqs=256, old_min=1, old_max=500, idle=3, lens=2),
        # a packed prefill of ragged prompts
        _case("append_prefill", "append", seqs=9, q_min=301, q_max=3001, layout="head", page_size=64, pad=5, lens=3),
        # small heads, rotated in part and in adjacent pairs, prompts resumed in mid-page
        _case("append_partial_rotation", "append", dtype="f16", heads=24, kv_heads=6, head_dim=64, seqs=33, q_min=1, q_max=129,
              old_min=0, old_max=333, rotary_dim=32, pairing="adjacent", page_size=32, lens=4),
        # one user's next token after a short conversation: latency
        _case("decode_one_user", "attend", dtype="f16", heads=12, kv_heads=12, old_min=977, old_max=977),
        # a serving batch with contexts of very different lengths
        _case("decode_long_ragged", "attend", heads=64, seqs=64, old_min=300, old_max=32000, idle=2, lens=5),
        # streaming generation: the last 1024 keys and the first 4 of long contexts
        _case("decode_window_sinks", "attend", seqs=128, old_min=500, old_max=9000, window=1024, sinks=4, layout="head",
              page_size=32, lens=6),
        # one long prompt from its first token
        _case("prefill_long", "attend", q_min=8192, q_max=8192, page_size=64),
        # packed ragged prompts under a window, 12 heads of 128 as in the attention shard
        _case("prefill_window_sinks", "attend", dtype="f16", heads=12, kv_heads=12, seqs=5, q_min=900, q_max=3500, window=1024,
              sinks=4, pad=7, lens=7),
        # pieces of long prompts next to single tokens of other users, small heads
        _case("chunked_prefill_mixed", "attend", heads=40, kv_heads=8, head_dim=64, seqs=12, q_min=1, q_max=700, old_min=2000,
              old_max=20000, layout="head", page_size=128, lens=8),
        # many samples of one long prompt, each with its own continuation
        _case("shared_prefix_decode", "shared", heads=32, seqs=128, old_min=0, old_max=600, prefix=12001, lens=9),
        # a few branches of one prompt that check a handful of proposed tokens each
        _case("shared_prefix_branches", "shared", dtype="f16", heads=16, kv_heads=16, head_dim=64, seqs=6, q_min=1, q_max=5,
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
        kv_heads, group = rng.choice([(12, 1), (16, 1), (8, 4), (8, 8), (4, 7), (8, 5), (6, 4), (2, 16), (1, 12)])
        head_dim = rng.choice([64, 128, 128])
        op = rng.choice(["append", "attend", "attend", "shared"])
        c = _case(None, op, dtype=rng.choice(["f16", "bf16"]), heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim,
                  page_size=rng.choice([16, 32, 64, 128]), layout=rng.choice(["token", "head"]), lens=rng.randrange(1 << 30),
                  pad=rng.choice([0, 0, 3]), rotary_dim=rng.choice([head_dim, head_dim, 32]), pairing=rng.choice(["half", "adjacent"]))
        if rng.random() < 0.5:  # single tokens, or a few each
            c["seqs"] = _log_int(rng, 1, 256)
            c["q_max"] = rng.choice([1, 1, 1, 4])
            c["old_max"] = _log_int(rng, 1, 32000)
            c["old_min"] = rng.randint(0, c["old_max"])
            c["idle"] = rng.choice([0, c["seqs"] // 8])
        else:  # prompts, whole or in pieces
            c["seqs"] = _log_int(rng, 1, 24)
            c["q_max"] = max(1, _log_int(rng, 24, 8192) // c["seqs"])
            c["q_min"] = rng.randint(1, c["q_max"])
            c["old_max"] = rng.choice([0, _log_int(rng, 1, 8000)])
        if op == "attend" and rng.random() < 0.5:
            c["window"] = _log_int(rng, 16, 4096)
            c["sinks"] = rng.choice([0, 1, 4, 130])
        if op == "shared":
            c["prefix"] = _log_int(rng, 100, 32000)
            c["old_max"] = min(c["old_max"], 1000)
            c["old_min"] = min(c["old_min"], c["old_max"])
        if _seconds(c) <= most and _cache_values(c) <= 2 ** 31:
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


def _cache_values(case):
    return _pages(case) * case["page_size"] * case["kv_heads"] * case["head_dim"]


def _seen(case, pos):
    """Keys that the query at position pos of its sequence sees."""
    if case["window"] <= 0 or pos < case["window"]:
        return pos + 1
    return case["window"] + min(case["sinks"], pos - case["window"] + 1)


def work(case):
    q, kv = _lengths(case)
    tokens, d, hq, hk = sum(q), case["head_dim"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        row = 2 * d * (hq + 2 * hk)
        return {"bytes": tokens * (2 * row + 4 * case["rotary_dim"]), "flops": tokens * (hq + hk) * case["rotary_dim"] * 3}
    keys = pairs = 0
    for n, m in zip(q, kv):
        if n == 0:
            continue
        first = m - n
        w = case["window"]
        keys += m if w <= 0 else m - max(0, first - w + 1) + min(case["sinks"], max(0, first - w + 1))
        if w <= 0:
            pairs += n * first + n * (n + 1) // 2
        else:
            pairs += sum(_seen(case, p) for p in range(first, m))
    if tokens:
        keys += case["prefix"]
        pairs += tokens * case["prefix"]
    return {"bytes": keys * hk * d * 2 * 2 + 2 * tokens * hq * d * 2, "flops": 4 * pairs * hq * d}


def prepare(case, seed):
    dt, dev = _DT[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    q, kv = _lengths(case)
    real, d, hq, hk, ps = sum(q), case["head_dim"], case["heads"], case["kv_heads"], case["page_size"]
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
    shape = (pages, ps, hk, d) if case["layout"] == "token" else (pages, hk, ps, d)

    def normal(*shape, size=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * size).to(dt)

    def cache():
        t = torch.empty(shape, device=dev, dtype=dt)
        for i in range(0, pages, 4096):
            t[i:i + 4096] = normal(*t[i:i + 4096].shape)
        return t

    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    s = {"case": case, "q": q, "kv": kv, "real": real, "tokens": tokens,
         "cu_q": torch.tensor(cu, dtype=torch.int32, device=dev), "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev),
         "table": table.to(dev), "prefix_table": order[:prefix_pages].to(dev), "k_cache": cache(), "v_cache": cache()}
    if case["op"] == "append":
        s["qkv"] = normal(tokens, (hq + 2 * hk) * d)
        s["q_out"] = torch.zeros(tokens, hq, d, device=dev, dtype=dt)
        r2 = case["rotary_dim"] // 2
        angle = torch.arange(max(kv) + 1, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(r2, dtype=torch.float64) / r2)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(dev)
    else:
        s["queries"] = normal(tokens, hq, d, size=1.5)
        s["out"] = torch.zeros(tokens, hq, d, device=dev, dtype=dt)
    if own:
        import consumer_gemm_chain_gb300 as cs
        desc = cs.cs_kv_desc_init(dtype=dt, heads=hq, kv_heads=hk, head_dim=d, page_size=ps, num_pages=pages,
                                  cache_layout=case["layout"], max_tokens=max(1, tokens), max_seqs=case["seqs"],
                                  rotary_dim=min(case["rotary_dim"], d), rotary_pairing=case["pairing"], window=case["window"],
                                  sinks=case["sinks"], shared=1 if case["op"] == "shared" else 0)
        s["plan"] = cs.cs_kv_plan(desc)
        s["batch"] = cs.cs_kv_batch(s["plan"], s["cu_q"], s["kv_lens"], s["table"], tokens=tokens, max_q=max(1, max(q)))
    return s


def run(s):
    if own:
        import consumer_gemm_chain_gb300 as cs
        op = s["case"]["op"]
        if op == "append":
            cs.cs_kv_append(s["plan"], s["batch"], s["qkv"], s["q_out"], s["k_cache"], s["v_cache"], rope=s["rope"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if op == "attend":
            cs.cs_kv_attention(s["plan"], s["batch"], s["queries"], s["k_cache"], s["v_cache"], s["out"])
        else:
            cs.cs_kv_attention_shared(s["plan"], s["batch"], s["queries"], s["k_cache"], s["v_cache"], s["prefix_table"],
                                      s["case"]["prefix"], s["out"])
        return s["out"]
    return _append(s) if s["case"]["op"] == "append" else _attend(s)


def _append(s):
    c, n = s["case"], s["real"]
    d, hq, hk, ps, rd = c["head_dim"], c["heads"], c["kv_heads"], c["page_size"], c["rotary_dim"]
    t = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    pos = s["kv_lens"].long()[seq] - s["cu_q"].long()[seq + 1] + t
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
    page, slot = s["table"].long()[seq, pos // ps], pos % ps
    kc, vc = s["k_cache"], s["v_cache"]
    if c["layout"] == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    kc[page, slot] = qk[:, hq:]
    vc[page, slot] = v.to(vc.dtype)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gather(cache, pages, count, layout):
    """The first `count` keys of the pages named, [kv_heads, count, head_dim] in 32 bits."""
    x = cache[pages.long()]
    x = x.permute(2, 0, 1, 3) if layout == "token" else x.permute(1, 0, 2, 3)
    return x.flatten(1, 2)[:, :count].float()


def _attend(s):
    c = s["case"]
    d, hq, hk, ps, w, prefix = c["head_dim"], c["heads"], c["kv_heads"], c["page_size"], c["window"], c["prefix"]
    group = hq // hk
    first = 0
    if prefix:
        k0 = _gather(s["k_cache"], s["prefix_table"], prefix, c["layout"])
        v0 = _gather(s["v_cache"], s["prefix_table"], prefix, c["layout"])
    for b, (n, m) in enumerate(zip(s["q"], s["kv"])):
        if n == 0:
            continue
        pages = s["table"][b, :-(-m // ps)]
        k, v = _gather(s["k_cache"], pages, m, c["layout"]), _gather(s["v_cache"], pages, m, c["layout"])
        if prefix:
            k, v = torch.cat([k0, k], 1), torch.cat([v0, v], 1)
        j = torch.arange(m + prefix, device="cuda")
        for i in range(0, n, 1024):
            e = min(n, i + 1024)
            x = s["queries"][first + i:first + e].float().view(e - i, hk, group, d).permute(1, 2, 0, 3)
            p = torch.arange(prefix + m - n + i, prefix + m - n + e, device="cuda")[:, None]
            hidden = j > p
            if w > 0:
                hidden = hidden | ((j <= p - w) & (j >= c["sinks"]))
            y = torch.empty(hk, group, e - i, d, device="cuda")
            for h in range(hk) if e - i > 64 else [slice(None)]:  # all heads at once where the scores are small
                z = x[h] @ k[h].transpose(-1, -2) if e - i > 64 else x @ k[:, None].transpose(-1, -2)
                z = (z * (1.0 / math.sqrt(d))).masked_fill(hidden, -math.inf)
                z = torch.exp(z - z.amax(-1, keepdim=True))
                z = z / z.sum(-1, keepdim=True)
                y[h] = z @ (v[h] if e - i > 64 else v[:, None])
            s["out"][first + i:first + e] = y.permute(2, 0, 1, 3).reshape(e - i, hq, d).to(s["out"].dtype)
        first += n
    return s["out"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    c = s["case"]
    d, hq, hk, ps, half = c["head_dim"], c["heads"], c["kv_heads"], c["page_size"], c["rotary_dim"] // 2
    q_out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    table, at = s["table"].cpu(), 0
    for b, (n, m) in enumerate(zip(s["q"], s["kv"])):
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
        for p in range((m - n) // ps, (m - 1) // ps + 1):
            a, e = max(p * ps, m - n), min(p * ps + ps, m)
            page = int(table[b, p])
            for cache, new in ((kc, qk[:, hq:]), (vc, rows[:, hq + hk:])):
                piece = new[a - (m - n):e - (m - n)]
                if c["layout"] == "token":
                    cache[page, a - p * ps:e - p * ps] = piece
                else:
                    cache[page, :, a - p * ps:e - p * ps] = piece.transpose(0, 1)
        at += n
    return q_out, kc, vc


def _exact_attend(s):
    c = s["case"]
    if work(c)["flops"] > 8e12:
        return None
    d, hk, ps, group, prefix = c["head_dim"], c["kv_heads"], c["page_size"], c["heads"] // c["kv_heads"], c["prefix"]
    out, at = s["out"].double(), 0
    spots = torch.arange(ps, device="cuda")
    shared = s["prefix_table"].long().repeat_interleave(ps) * ps + spots.repeat(len(s["prefix_table"]))
    for b, (n, m) in enumerate(zip(s["q"], s["kv"])):
        if n == 0:
            continue
        # each key's row of the cache, the shared prefix first, and its place in the sequence
        cols = -(-m // ps)
        where = torch.cat([shared[:prefix], (s["table"][b, :cols].long().repeat_interleave(ps) * ps + spots.repeat(cols))[:m]])
        place = torch.arange(len(where), device="cuda")
        for h in range(hk):
            if c["layout"] == "token":
                k, v = (s[x].view(-1, hk, d)[where, h].double() for x in ("k_cache", "v_cache"))
            else:
                page, spot = where // ps, where % ps
                k, v = (s[x][page, h, spot].double() for x in ("k_cache", "v_cache"))
            for i in range(0, n, 256):
                e = min(n, i + 256)
                x = s["queries"][at + i:at + e, h * group:(h + 1) * group].double()
                score = torch.einsum("tgd,kd->tgk", x, k) / d ** 0.5
                back = (torch.arange(i, e, device="cuda") + len(where) - n)[:, None] - place[None]  # how far the key lies behind
                seen = back >= 0
                if c["window"] > 0:
                    seen &= (back < c["window"]) | (place < c["sinks"])[None]
                score = torch.where(seen[:, None], score, float("-inf"))
                weight = torch.exp(score - torch.logsumexp(score, -1, keepdim=True))
                out[at + i:at + e, h * group:(h + 1) * group] = torch.einsum("tgk,kd->tgd", weight, v)
        at += n
    return out
