"""The attention workloads of bench.py carry metrics of their own, and the default stays."""
import inspect
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


def test_attention_workloads_have_their_own_metrics():
    assert set(bench.METRICS_ATTEND) == {"attend", "decode"}
    assert len({bench.METRIC, *bench.METRICS_I8.values(), *bench.METRICS_ATTEND.values()}) == 5
    source = inspect.getsource(bench.run_attend)
    assert "METRICS_ATTEND[args.workload]" in source and '"metric": METRIC,' not in source


def test_default_workload(monkeypatch):
    monkeypatch.setattr(sys, "argv", ["bench.py"])
    assert bench.parse().workload == "proj"
