"""The benchmark's one line: short enough that the last 8000 characters of its output hold
it, with every key of the full record's top level and the headline workload untouched."""

import json

import bench

X = 1234.5678901234567


def _record():
    kernel = dict(kernel="fno_fwd_plane_mx", launch_shape="separate", ms=X, algorithmic_bytes=10 ** 9, exchange_bytes=10 ** 8, gbps=X,
                  frac=X / 1e4, gbps_with_exchange=X)
    roof = dict(bound="hbm", kernel="fno_fwd_plane_mx", achieved=X, peak=8000.0, unit="GB/s", frac=X / 1e4, traffic=10 ** 9,
                algorithmic_bytes=10 ** 9, exchange_bytes=10 ** 8, ms_per_launch=X, achieved_with_exchange=X)
    stat = dict(mean=X, std=X, min=X, p50=X, p99=X)
    cpu = dict(value=X, unit="layers/s", cores=16, kind="oracle", sample="s" * 220, gbps_minimal_bytes=X)
    work = dict(workload="c2", description="d" * 80, dtype="bf16", ms_per_layer=X, layers_per_s=X, minimal_bytes=10 ** 9, gbps=X,
                hbm_frac=X / 1e4, per_layer_us=stat, hot_single_set_layers_per_s=X, launch_shape="separate", half_exchange=True,
                arithmetic="a" * 280, launch_shapes={k: dict(ms_per_layer=X, layers_per_s=X, launches_per_layer=3)
                                                     for k in ("fused", "separate")}, kernels=[kernel] * 5, roofline=roof)
    out = dict(metric=bench.METRIC, value=X, unit="layers/s", n_gpus=1, steps=20, warmup=5, ms_per_step=X, higher_is_better=True,
               scaling="weak", vs_baseline=None, dtype="f16", arithmetic="a" * 280, data="d" * 60,
               config=dict(workload="w" * 70, grid=[256, 256], storage="f16"), gbps=X, hbm_frac=X / 1e4, roofline=roof,
               kernels=[kernel] * 3, per_layer_us=stat, hot_single_set_layers_per_s=X, settle_ms=300.0, cpu_baseline=cpu)
    out["metric_configs"] = [dict(work, cpu_baseline=cpu, dtype_label="l" * 22, steps=200) for _ in bench.METRIC_CONFIGS]
    out["configs"] = [dict(work, steps=200)]
    out["backward"] = [{f"quantity_{i:02d}_of_bwd": X for i in range(14)}] * 3
    out["model"] = dict({f"quantity_{i}": X for i in range(5)}, latency_b1_us=stat, latency_b1_graph_us=stat)
    sweep = dict(batch=1, launch_shape="separate", eager_us=stat, eager_fused_us=stat, graph_us=stat, samples_per_s_eager=X,
                 samples_per_s_graph=X)
    out["latency"] = dict(workload="w" * 70, calls_per_batch=200, sweep=[sweep] * 4, throughput_gain_b1_to_b8_eager=X)
    out["copy_1gib"] = dict(bytes_copied=1 << 31, ms=X, gbps=X)
    return out


def test_line_is_short_and_whole():
    out = _record()
    text = json.dumps(bench.short_line(out), separators=(",", ":"))
    assert len(text) < 7500 < len(json.dumps(out))
    line = json.loads(text)
    assert set(line) == set(out)
    assert line["value"] == X and line["ms_per_step"] == X and line["metric"] == bench.METRIC
    for k in ("unit", "n_gpus", "steps", "warmup", "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "config"):
        assert line[k] == out[k]
    assert line["roofline"].keys() == out["roofline"].keys() and abs(line["roofline"]["frac"] / (X / 1e4) - 1) < 1e-5
    assert len(line["metric_configs"]) == len(bench.METRIC_CONFIGS)
    for w in line["metric_configs"]:
        assert abs(w["layers_per_s"] / X - 1) < 1e-5 and w["roofline"]["traffic"] == 10 ** 9 and w["cpu_baseline"]["cores"] == 16


def test_line_of_a_run_without_the_extras():
    out = {k: v for k, v in _record().items() if k not in ("latency", "model", "backward", "cpu_baseline")}
    out["metric_configs"] = [dict(out["configs"][0], cpu_baseline=None)]
    assert bench.short_line(out)["metric_configs"][0]["cpu_baseline"] is None
