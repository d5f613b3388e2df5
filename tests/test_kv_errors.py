"""Errors of the CUDA runtime that the paged cache calls report."""
import kv_programs


def test_a_reported_error_is_not_left_behind(tmp_path):
    assert kv_programs.run("kv_error_check", tmp_path) == (0, "ok")
