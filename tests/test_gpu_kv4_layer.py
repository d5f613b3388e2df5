"""An attention layer over the cache in 4 bits (cs_attn_cached4_forward) in both types."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import consumer_gemm_chain_gb300 as cs
import oracle
from kv_util import rope_table
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("steps", [[1], [150, 1, 3], [20, 40, 1]])
def test_steps_of_two_sequences(dtype, layout, steps):
    """Steps of `steps` tokens, shared out to two sequences (one of them of no tokens at times): outputs over what the cache holds
    then, which a reading gives. Within ten roundings of the dtype: X Wqkv, the rotation, scores of two rounded factors (twice in
    a softmax), weights, O, Y, and two for sums."""
    H, heads = 256, 2
    F, total = heads * 128, sum(steps)
    g = torch.Generator().manual_seed(total)
    X = (torch.randn(total, H, generator=g) * 0.5).to(dtype)
    Wqkv = (torch.randn(H, 3 * F, generator=g) * 0.06).to(dtype)
    Wo = (torch.randn(F, H, generator=g) * 0.06).to(dtype)
    rope = rope_table(total, 128).cuda()
    plan = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=heads, num_pages=40, max_tokens=total, max_seqs=2,
                                            rotary_dim=128, cache_layout=layout))
    codes, scales = cs.cs_kv4_shapes(plan)
    k, v = ((torch.full(codes, 0x5A, dtype=torch.uint8, device="cuda"), torch.full(scales, 0xFF, dtype=torch.uint8, device="cuda"))
            for _ in range(2))
    table = torch.randperm(40, generator=g)[:24].to(torch.int32).view(2, 12).cuda()
    lens, at = [0, 0], 0
    for n in steps:
        new = [n - n // 3, n // 3]
        lens = [a + b for a, b in zip(lens, new)]
        cu = torch.tensor([0, new[0], n], dtype=torch.int32, device="cuda")
        kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
        batch = cs.cs_kv_batch(plan, cu, kv, table, tokens=n, max_q=max(new))
        x = X[at:at + n]
        Y = torch.full((n, H), 7.0, dtype=dtype, device="cuda")
        desc = cs.cs_chain_desc_init(kind="attn", M=n, H=H, F=F, dtype=dtype, heads=heads, head_dim=128, split_k=1, sk_tiles=-1)
        with cs.cs_chain_plan(desc) as chain:
            cs.cs_attn_cached4_forward(chain, plan, batch, x.cuda(), Wqkv.cuda(), Wo.cuda(), Y, k, v, rope=rope)
            torch.cuda.synchronize()
            assert cs.cs_chain_status(chain) == cs.CS_OK and cs.cs_kv_status(plan) == cs.CS_OK
        # what the cache holds, sequence after sequence
        m = sum(lens)
        whole = cs.cs_kv_plan(cs.cs_kv_desc_init(dtype=dtype, heads=heads, kv_heads=heads, num_pages=40, max_tokens=m, max_seqs=2,
                                                 cache_layout=layout))
        rows = cs.cs_kv_batch(whole, torch.tensor([0, lens[0], m], dtype=torch.int32, device="cuda"), kv, table, tokens=m, max_q=m)
        K, V = (torch.empty(m, heads, 128, dtype=dtype, device="cuda") for _ in range(2))
        cs.cs_kv4_read(whole, rows, k, v, K, V)
        torch.cuda.synchronize()
        K, V = okv.to64(K), okv.to64(V)
        pos = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, new)])
        t = okv.to64(rope.cpu())[pos][:, None]
        qkv = (okv.to64(x) @ okv.to64(Wqkv)).reshape(n, 3 * heads, 128)
        q = okv.rotate(qkv[:, :heads], t[..., :64], t[..., 64:], "half")
        O = np.zeros((n, heads, 128))
        for i in range(n):
            s = int(i >= new[0])
            own = slice(0, lens[0]) if s == 0 else slice(lens[0], m)
            for h in range(heads):
                O[i, h] = okv.attend(q[i, h], K[own, h], V[own, h], okv.visible(pos[i], lens[s], 0, 0), 128 ** -0.5)[0]
        assert oracle.rel_err(Y.cpu(), O.reshape(n, F) @ okv.to64(Wo)) <= 10 * torch.finfo(dtype).eps / 2
        # the new keys are within a little more than half a step of the exact ones (and of their own rounding)
        exact = okv.rotate(qkv[:, heads:2 * heads], t[..., :64], t[..., 64:], "half")
        step = np.abs(exact).reshape(n, heads, 4, 32).max(-1).repeat(32, -1) / 7
        held = np.concatenate([K[lens[0] - new[0]:lens[0]], K[m - new[1]:m]])
        assert (np.abs(held - exact) <= 0.6 * step + 4 * torch.finfo(dtype).eps * np.abs(exact).max()).all()
        at += n
