"""bench.py's line of JSON stays short enough for a log to keep it whole."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


def _entry(workload, mask, form, chunk):
    third = 1 / 3
    roof = {"bound": "hbm", "achieved": third, "peak": 6675.8, "unit": "GB/s", "frac": third, "algorithmic_bytes": 1 << 30}
    return {"workload": f"{workload} B=64 H=12 L=24337 d=64", "mask": mask, "form": form, "chunk": chunk,
            "input_dtype": "bf16", "value": third * 1e9, "unit": "tokens/s", "ms_per_step": third, "steps": 20,
            "launches_per_call": 2, "path": "tcgen05 chunk-128 (pre-pass, main pass)", "roofline": roof, "hbm": roof,
            "cpu_baseline": {"value": third, "unit": "tokens/s", "cores": 16, "kind": "oracle", "sample": "x" * 200}}


def test_line_is_short_and_whole():
    line = {"metric": bench.METRIC, "value": 1e9 / 3, "n_gpus": 1, "vs_baseline": None, "roofline": {"traffic": None},
            "configs": [_entry(*c) for c in bench.CONFIG_LINES]}
    text = bench.short_line(line)
    assert "\n" not in text and len(text) < 9000   # the rest of a whole run's line is 5.5 KB
    got = json.loads(text)
    assert set(got) == set(line) and abs(got["value"] / line["value"] - 1) < 1e-6
    assert [(c["workload"].split()[0], c["mask"], c["form"], c["chunk"]) for c in got["configs"]] \
        == [tuple(c) for c in bench.CONFIG_LINES]
    assert all(c["ms_per_step"] and c["roofline"]["frac"] and c["launches_per_call"] == 2 for c in got["configs"])
    assert json.loads(bench.short_line(dict(line, configs=None)))["configs"] is None
