"""Refusals of cs_attn_cached_forward without a GPU."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

import kv_programs


@pytest.fixture(scope="module")
def cs():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import consumer_gemm_chain_gb300 as cs
    return cs


def test_refusals_come_before_any_work(tmp_path):
    assert kv_programs.run("kv_layer_check", tmp_path) == (0, "ok")


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


@pytest.mark.parametrize("which", range(4))
def test_tensors_of_another_device_are_refused(cs, which):
    chain = SimpleNamespace(handle=None, desc=cs.cs_chain_desc_init(kind="attn", M=3, H=256, F=256, heads=2, head_dim=128))
    shapes = [(3, 256), (256, 768), (256, 256), (3, 256)]
    tensors = [torch.zeros(s, dtype=torch.float16).as_subclass(OnDevice) for s in shapes]
    tensors[which].index = 1
    plan = SimpleNamespace(handle=None, device=0, dtype=torch.float16, cache_shape=(1, 16, 2, 128),
                           _append=cs.kv.cs_kv_append_args())
    batch = cs.KVBatch(cs.kv.cs_kv_batch_s(tokens=3), (), 0)
    cache = torch.zeros(plan.cache_shape, dtype=torch.float16).as_subclass(OnDevice)
    with pytest.raises(ValueError, match=["X", "Wqkv", "Wo", "Y"][which] + ".*cuda:1"):
        cs.cs_attn_cached_forward(chain, plan, batch, *tensors, cache, cache, stream=0)
