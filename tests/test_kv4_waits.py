"""The limits of the waits inside the tensor-core kernel over a cache in 4 bits."""
from __future__ import annotations

import pytest

import kv_programs


@pytest.mark.gpu
def test_kernels_whose_waits_run_out(tmp_path):
    """Every wait runs out at once: the calls end, the outputs are left alone, the status says so, and a
    reset clears it."""
    assert kv_programs.run("kv4_give_up_check", tmp_path, device=True) == (0, "ok")
