"""Which factors of the scores a plan of the paged cache takes, without a GPU."""
from __future__ import annotations

import numpy as np
import pytest


@pytest.fixture(scope="module")
def cs():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import consumer_gemm_chain_gb300 as cs
    return cs


def refusal(cs, scale):
    desc = cs.cs_kv_desc_init(heads=2, kv_heads=2, num_pages=4, max_tokens=8, max_seqs=2, scale=float(scale))
    try:
        cs.cs_kv_destroy(cs.cs_kv_plan(desc))
    except cs.CSError as e:
        return "scale" in str(e)
    return False


def test_scales(cs):
    """The kernels multiply by scale * log2(e) in 32 bits, which has to be finite."""
    largest = np.finfo(np.float32).max
    for scale in (largest, largest / np.float32(1.4426)):
        assert refusal(cs, scale)
    for scale in (largest / np.float32(1.4428), 1.0, 0.0, np.finfo(np.float32).tiny):
        assert not refusal(cs, scale)
