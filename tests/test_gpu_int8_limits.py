"""More rows than one launch can hold: a launch's threads are counted in 32
bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


def _around(n, *borders):
    """Runs of rows at the ends of n rows and around the borders."""
    return [(0, 40), (n - 40, n)] + [(b - 20, min(n, b + 20)) for b in borders]


@pytest.mark.parametrize("nt,id_,ld,border", [((1 << 26) + 77, 4, 4, 1 << 26), ((1 << 24) + 77, 513, 513, 1 << 24)])
def test_quantize_many_rows(qig, nt, id_, ld, border):
    """One row a wave and one row a workgroup of 256, over 2^32 threads each."""
    print("quantize_i8", nt, id_, flush=True)
    x = torch.empty((nt, ld), dtype=torch.bfloat16, device="cuda")[:, :id_]
    x.normal_()
    s = torch.full((nt,), -1.0, device="cuda")
    q, _ = qig.quantize_i8(x, s=s)
    assert bool((s > 0).all()), "rows left out"
    for lo, hi in _around(nt, border, border // 2):
        q1, s1 = qig.quantize_i8(x[lo:hi].clone())
        assert torch.equal(q[lo:hi], q1) and torch.equal(s[lo:hi], s1), lo


def test_route_many_tokens(qig):
    nt = (1 << 26) + 77
    print("route_experts", nt, flush=True)
    l = torch.empty((nt, 3), dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.full((nt, 2), -7, dtype=torch.int32, device="cuda")
    _, w = qig.route_experts(l, 2, ids=ids)
    assert bool((ids >= 0).all()), "tokens left out"
    for lo, hi in _around(nt, 1 << 26, 1 << 25):
        i1, w1 = qig.route_experts(l[lo:hi].clone(), 2)
        assert torch.equal(ids[lo:hi], i1) and torch.equal(w[lo:hi], w1), lo


def test_combine_many_tokens(qig):
    """Three threads a token, over 2^32 of them: 52 GB in."""
    nt, od = (1 << 32) // 3 + 77, 9
    print("combine_experts", nt, od, flush=True)
    h = torch.empty((nt, od), device="cuda").normal_()
    w = torch.rand((nt, 1), device="cuda")
    y = torch.full((nt, od), float("nan"), dtype=torch.bfloat16, device="cuda")
    qig.combine_experts(h, w, y=y)
    assert not bool(torch.isnan(y).any()), "tokens left out"
    border = (1 << 32) // 3
    for lo, hi in _around(nt, border, border // 2):
        assert torch.equal(y[lo:hi], qig.combine_experts(h[lo:hi].clone(), w[lo:hi].clone(), dtype=torch.bfloat16)), lo


def test_product_many_weight_rows(qig):
    """One token and 2^27 and more weight rows of 16 bytes: more than the
    few-token kernel's launch holds."""
    od = (1 << 27) + 77
    print("mm_i8", od, flush=True)
    W = torch.randint(-128, 128, (od, 16), dtype=torch.int8, device="cuda")
    sw = torch.rand(od, device="cuda")
    q = torch.randint(-127, 128, (1, 16), dtype=torch.int8, device="cuda")
    sq = torch.rand(1, device="cuda")
    y = torch.full((1, od), float("nan"), device="cuda")
    qig.mm_i8(W, sw, q, sq, y=y)
    assert not bool(torch.isnan(y).any()), "outputs left out"
    for lo, hi in _around(od, 1 << 27, 1 << 26):
        want = (W[lo:hi].double() @ q[0].double()) * sq.double() * sw[lo:hi].double()
        # the sum is exact in fp32, two products round by 2^-24 each
        assert bool(((y[0, lo:hi].double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()), lo
