"""Arguments that overlap, without a GPU."""
import kv_programs


def test_overlapping_arguments(tmp_path):
    assert kv_programs.run("kv_overlap_check", tmp_path) == (0, "ok")
