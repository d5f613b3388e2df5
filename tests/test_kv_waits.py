"""The limits of the waits inside the attention kernels over the paged cache."""
from __future__ import annotations

import pytest

import kv_programs


def test_limits_of_the_waits_on_the_host(tmp_path):
    assert kv_programs.run("kv_wait_check", tmp_path) == (0, "ok")


@pytest.mark.gpu
def test_kernels_whose_waits_run_out(tmp_path):
    """Every wait runs out at once, with copies on their way: the calls end, the outputs are left
    alone, the status says so, and a reset clears it."""
    assert kv_programs.run("kv_give_up_check", tmp_path, device=True) == (0, "ok")


def test_an_item_begins_when_its_queries_are_there(tmp_path):
    assert kv_programs.run("kv_query_phase_check", tmp_path) == (0, "ok")
