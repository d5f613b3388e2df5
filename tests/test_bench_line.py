"""The bench's line stays short: other workloads in four numbers a row, in full in a file."""
import json

import bench


def record(m, key):
    whole = {"span_us": 68.06412345678, "busy_frac": 0.5985109989359859, "tail_us": 43.55212345678, "sms_used": 152}
    return {"M": m, "plan": {"tile_m": 128, "tile_n": 128, "splits": [2, 2], "tuned_entry": 39}, f"{key}_us": 72.40608215332031,
            "strided_us": 73.38367938995361, "stream_us": 75.80863952636719, "roofline_frac": 0.4567891234, "bound": "hbm",
            "tail": {p: {"launches": [whole] * 2, "whole": whole} for p in ("tile", "stream")}}


def test_short_configs():
    full = {"llama_swiglu": [record(m, "tile") for m in range(7)], "attention_chain": [record(m, "row") for m in range(7)],
            "stress": [record(m, "tile") for m in range(12)], "with_nothing": []}
    short = bench.short_configs(full)
    assert list(short) == list(full)
    assert short["attention_chain"][3] == {"M": 3, "us": 72.41, "control_us": 75.81, "roofline_frac": 0.4568}
    assert len(json.dumps(short)) < 2500 < len(json.dumps(full))


def test_details_go_to_the_file_only(tmp_path):
    line = {"value": 1.0, "extras": {"sweep": [], "other_configs": {"stress": [record(128, "tile")]}}}
    path = tmp_path / "details.json"
    out = bench.shortened(line, str(path))
    assert json.loads(path.read_text()) == line
    assert out["extras"]["other_configs"] == bench.short_configs(line["extras"]["other_configs"]) and out["extras"]["sweep"] == []
    assert bench.shortened(line, None) == out
    assert bench.shortened({"value": 2.0}, None) == {"value": 2.0}
