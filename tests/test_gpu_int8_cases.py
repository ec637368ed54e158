"""The experts' down case of perf/operators.py, as its calls run it, against
its 64-bit form."""
import importlib.util
import os

import numpy as np
import pytest

import int8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


@pytest.mark.parametrize("y", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nt,e,k,od,id_", [(37, 5, 3, 200, 130), (300, 8, 6, 257, 1000)])
def test_down_case_is_rounded_once(ops, nt, e, k, od, id_, y):
    """The rows' sum is rounded to the output's type once: the rows before it
    are not.  A row's value takes two fp32 products (its sum of at most 1000
    products of int8 is below 2^24), the weighted sum k products and k
    additions, each off by at most 2^-24 of a value no larger than the sum of
    the magnitudes, and the output half a step of its type."""
    c = {"op": "down", "nt": nt, "e": e, "k": k, "od": od, "id": id_, "x": "bf16", "y": y}
    print("down case", c, flush=True)
    state = ops.prepare(c, 3)
    got = ops.run(state)
    assert got.dtype == ops.TYPES[y]
    want = ops.exact(c, 3)
    rows = ops._exact_experts(state["x"], state["w"], state["sw"], state["ids"], False)
    size = (rows.abs().view(nt, k, od) * state["rw"].double()[:, :, None]).sum(1)
    kind = str(got.dtype).split(".")[1]
    d = (2 * k + 3) * 2.0 ** -24 * size
    allow = d + ref.EPS[kind] * (want.abs() + d) + ref.FLOOR[kind]
    err = ((got.double() - want).abs() / allow).max().item()
    print("of the allowance", err, flush=True)
    assert np.isfinite(err) and err <= 1.0
