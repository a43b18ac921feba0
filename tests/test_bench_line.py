"""The benchmark's printed line: short enough that what keeps only the end of a
run's output keeps all of it, with every key of the contract."""
import json
import types

import bench
from rotated_bit_post_b200 import inputs


def _record():
    args = bench.parse(["--steps", "20", "--warmup", "5", "--no-cpu-baseline"])
    clocks = {"sm_mhz": 1785.123456789, "sm_max_mhz": 1965.0, "reasons": ["sw_power_cap"], "samples": 1234,
              "source": "nvml, 1 ms period, during the timed steps"}
    res = {}
    for n in bench.ORDER:
        w = inputs.workload(n)
        t = [0.1234567890123456] * 20
        res[n] = bench.layer_result(types.SimpleNamespace(w=w, dev="cpu"), args, t, t, t, clocks, None, 1, 148)
        res[n]["bf16_linear"] = {"ms": 0.03777599968016147, "tflops": 1151.1685789969308, "what": "x" * 200}
        res[n]["speedup_vs_bf16_linear"] = 0.3471395111820079
        res[n]["e2e"] = {"value": 5637400.672542427, "unit": "tokens/s", "h2d_bytes_per_step": 9437184,
                         "d2h_bytes_per_step": 1174118400, "ms_per_step": 0.7265759944915772, "steps": 20, "note": "x" * 200}
    out = bench.record(args, bench.ORDER, res, 1)
    out["cpu_baseline"] = {"value": 3708.672483781052, "unit": "tokens/s", "cores": 128, "kind": "oracle", "sample": "x" * 200}
    return out


def test_line_is_short_and_whole():
    out = _record()
    line = json.dumps(bench.short_line(out))
    assert len(line) <= bench.LINE_MAX, len(line)
    got = json.loads(line)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "clocks", "e2e", "gpu_launches", "roofline", "cpu_baseline"):
        assert key in got, key
    assert abs(got["value"] / out["value"] - 1) < 1e-8 and abs(got["ms_per_step"] / out["ms_per_step"] - 1) < 1e-8
    assert got["e2e"]["h2d_bytes_per_step"] == 9437184 and got["e2e"]["unit"] == "tokens/s"
    assert got["clocks"]["reasons"] == ["sw_power_cap"]
    assert set(got["configs"]) == set(bench.ORDER)
    assert got["config"] == out["config"]


def test_full_record_was_longer():
    # what the line leaves out is in the record that --details writes
    assert len(json.dumps(_record())) > 2 * bench.LINE_MAX
