"""bench.py's modes on the GPU, with few steps."""
import json
from types import SimpleNamespace

import pytest

pytestmark = pytest.mark.gpu


def test_cache_mode(gpu_lib, capsys):
    """One JSON line of the 8-bit cache's mode: its value follows from the
    time of a step, its rate from the bytes and the attention's time."""
    import bench
    bench.cache_bench(SimpleNamespace(steps=3, warmup=2, ramp_seconds=0.0))
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 1
    line = json.loads(lines[0])
    cfg = line["config"]
    assert line["n_gpus"] == 1 and line["steps"] == 3 and line["warmup"] == 2 and line["ramp_steps"] == 2
    assert line["data"] == "synthetic" and line["dtype"] == "bf16" and line["higher_is_better"] is True
    assert line["value"] == pytest.approx(cfg["B"] * cfg["N"] / line["ms_per_step"] * 1e3)
    # at least 1001 tokens of K and V a sequence are read
    assert line["bytes_per_attention"] > cfg["B"] * 1001 * 2 * cfg["heads"] * cfg["dim"]
    assert line["hbm_gbps"] == pytest.approx(line["bytes_per_attention"] / line["attention_us"] / 1e3)
    assert 0 < line["hbm_frac_of_peak"] < 1 and line["append_us"] > 0
