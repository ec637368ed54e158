"""The gated activation of the int8 products, apart from the products' own
roundings: one weight and one activation of 1, so that the gate's value is the
weight's scale itself and the other factor 1."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


# one token and few: the register kernel; more: tiles
@pytest.mark.parametrize("nt", [1, 100])
def test_gate_keeps_its_digits_far_from_zero(qig, nt):
    """In units of u = 2^-24, relative: exp2 within an ulp 2, the correction
    for its rounded argument 1, their product 1, the sum with 1 1, the
    reciprocal within an ulp 2, two products 2 and the correction's
    neglected square below 1: 10 whatever the value is.  Where the exponential
    passes 2^126 its reciprocal is below the smallest normal number: 2^-119
    covers 88.8 times that."""
    g = np.random.Generator(np.random.PCG64([20261, nt]))
    a = np.concatenate([np.linspace(-90, 90, 3001), g.standard_normal(3000) * 3, -20 - g.random(500), 1e-30 * g.random(20),
                        [0.0, -0.0, -100.0, -1e4, -3e38, 100.0, 1e4, 3e38]]).astype(np.float32)
    od = len(a)
    W = torch.zeros((2 * od, 16), dtype=torch.int8)
    W[:, 0] = 1
    q = torch.zeros((nt, 16), dtype=torch.int8)
    q[:, 0] = 1
    sw = np.concatenate([a, np.ones(od, np.float32)])
    y = qig.mm_i8(W.cuda(), torch.from_numpy(sw).cuda(), q.cuda(), torch.ones(nt, device="cuda"), glu=True)
    x = a.astype(np.float64)
    with np.errstate(over="ignore"):
        want = x / (1 + np.exp(-x))
    got = y.cpu().numpy().astype(np.float64)
    err = np.abs(got - want) / (10 * 2.0 ** -24 * np.abs(want) + 2.0 ** -119)
    worst = err.max(0)
    print("worst", worst.max(), "at", a[worst.argmax()], flush=True)
    assert np.isfinite(got).all() and worst.max() <= 1.0


@pytest.mark.parametrize("nt", [1, 100])
def test_gate_of_extreme_values(qig, nt):
    """Infinities and NaN go through as a * sigmoid(a) * b has them."""
    inf = float("inf")
    a = torch.tensor([inf, 3e38, 2.4e38, 128.0, 128.5, float("nan"), -128.0, -2e38, -3.4e38, 0.0])
    od = len(a)
    W = torch.zeros((2 * od, 16), dtype=torch.int8)
    W[:, 0] = 1
    q = torch.zeros((nt, 16), dtype=torch.int8)
    q[:, 0] = 1
    y = qig.mm_i8(W.cuda(), torch.cat([a, torch.ones(od)]).cuda(), q.cuda(), torch.ones(nt, device="cuda"), glu=True)
    want = torch.where(a < -100, torch.zeros(()), a).expand(nt, od)
    got = y.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
