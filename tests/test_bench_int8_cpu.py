"""The int8 workloads of bench.py carry metrics of their own."""
import inspect
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


def test_int8_workloads_are_not_labelled_as_k_quant_gemms():
    assert set(bench.METRICS_I8) == {"ffn_i8", "experts"}
    assert len({bench.METRIC, *bench.METRICS_I8.values()}) == 3
    for m in bench.METRICS_I8.values():
        assert "_K" not in m and "TOPS" in m
    source = inspect.getsource(bench.run_int8)
    assert "METRICS_I8[args.workload]" in source and '"metric": METRIC,' not in source
