"""The int8 linear layer and the experts' operators on the GPU against plain
64-bit forms (int8_ref)."""
import numpy as np
import pytest

import int8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


def _rng(*key):
    return np.random.Generator(np.random.PCG64([20260, *key]))


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _say(*a):
    print(*a, flush=True)


def _rows(a, ld, fill=99):
    """a [rows][n] on the GPU as a view of rows of ld elements, the rest of
    each row holding `fill`."""
    p = torch.full((a.shape[0], ld), fill, dtype=a.dtype)
    p[:, :a.shape[1]] = a
    return p.cuda()[:, :a.shape[1]]


# --- quantization -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("nt,id_", [(1, 1), (1, 7), (3, 8), (2, 63), (5, 64), (2, 255), (4, 256), (3, 1000), (2, 1025),
                                    (7, 3584), (2, 4099), (3, 18944), (1, 40000), (300, 129)])
def test_quantize_rows(qig, kind, nt, id_):
    g = _rng(1, nt, id_)
    x = torch.from_numpy(g.standard_normal((nt, id_)).astype(np.float32) * 3).to(TYPES[kind])
    _say("quantize_i8", kind, nt, id_)
    q, s = qig.quantize_i8(x.cuda())
    assert q.shape == (nt, id_) and q.stride(0) % 16 == 0
    rq, rs = ref.quantize(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quantize_borders_and_extremes(qig):
    """Values at the border between two integers and next to it, the ends of
    the number range, zeros; all decided as the exact quotient is."""
    one = np.float32(1)
    rows = []
    for amax in (127.0, 1.0, 3.3333333, 1e-38, 1.4e-45 * 200, 1.4e-45 * 190, 1.4e-45 * 30, 3.4e38, 1e30, 5.877e-39):
        amax = np.float32(amax)
        s = np.float64(amax / np.float32(127))
        mid = ((np.arange(32) * 4 + 0.5) * s).astype(np.float32)
        row = np.concatenate([mid, np.nextafter(mid, one * 0), np.nextafter(mid, np.float32(np.inf)), [0, -0.0]])
        row = np.where(np.arange(len(row)) % 2, -row, row).astype(np.float32)
        rows.append(np.clip(np.concatenate([row, [amax]]), -amax, amax).astype(np.float32))
    x = np.stack(rows + [np.zeros_like(rows[0])])
    _say("quantize_i8 borders", x.shape)
    q, s = qig.quantize_i8(torch.from_numpy(x).cuda())
    rq, rs = ref.quantize(x)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_rows_with_nan_or_infinity(qig, kind):
    x = torch.ones(4, 300)
    x[0, 7], x[1, 299], x[2, 0] = float("nan"), float("inf"), float("-inf")
    q, s = qig.quantize_i8(x.to(TYPES[kind]).cuda())
    assert torch.isnan(s[:3]).all() and (q[:3] == 0).all()
    assert (q[3] == 127).all()
    W, sw = qig.quantize_i8(torch.ones(2, 300).cuda())
    y = qig.mm_i8(W, sw, q, s)
    assert torch.isnan(y[:3]).all() and torch.isfinite(y[3]).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("off,ldx,id_", [(0, 80, 64), (1, 81, 64), (3, 77, 70), (8, 96, 33), (0, 4200, 4100)])
def test_quantize_strides_and_guards(qig, kind, off, ldx, id_):
    """Views that start and step at any element; nothing but the rows' own
    bytes is written."""
    g = _rng(2, off, ldx)
    base = torch.from_numpy(g.standard_normal(9 * ldx + off).astype(np.float32)).to(TYPES[kind])
    x = torch.as_strided(base.cuda(), (9, id_), (ldx, 1), off)
    q = torch.full((11, id_ + 29), 55, dtype=torch.int8, device="cuda")
    s = torch.full((11,), 55.0, device="cuda")
    qig.quantize_i8(x, q=q[1:10, 13:13 + id_], s=s[1:10])
    rq, rs = ref.quantize(torch.as_strided(base, (9, id_), (ldx, 1), off).float().numpy())
    want = np.full((11, id_ + 29), 55, np.int8)
    want[1:10, 13:13 + id_] = rq
    assert np.array_equal(q.cpu().numpy(), want)
    assert s[0] == 55 and s[10] == 55 and np.array_equal(s[1:10].cpu().numpy(), rs)


# --- product ------------------------------------------------------------------------------------------------

def _operands(g, nt, rows, id_, bias):
    q = g.integers(-127, 128, (nt, id_)).astype(np.int8)
    W = g.integers(-128, 128, (rows, id_)).astype(np.int8)
    sq = (g.random(nt) * 0.02 + 1e-3).astype(np.float32)
    sw = (g.random(rows) * 0.02 + 1e-4).astype(np.float32)
    # outputs of order one, as after a quantization
    sq /= np.float32(max(1.0, np.sqrt(id_) / 4))
    b = g.standard_normal(rows).astype(np.float32) if bias else None
    return q, W, sq, sw, b


def _pad(n, extra=0):
    return (n + 15) // 16 * 16 + 16 * extra


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _check(y, want, allow, what):
    err = np.abs(_np(y) - want)
    assert np.isfinite(_np(y)).all(), what
    worst = float((err / allow).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"


SIZES = [(1, 1, 1), (1, 3, 16), (2, 17, 15), (5, 16, 17), (15, 64, 128), (16, 33, 127), (17, 128, 129), (31, 100, 256),
         (33, 256, 64), (48, 127, 640), (64, 129, 383), (65, 255, 1000), (100, 31, 2049), (127, 300, 130),
         (128, 128, 512), (129, 257, 96), (200, 512, 257), (256, 256, 384), (257, 130, 1023), (300, 700, 113),
         (520, 520, 512), (1, 3584, 3584), (7, 1030, 5003), (1000, 64, 300), (70, 2100, 1100)]


@pytest.mark.parametrize("ytype", list(TYPES))
@pytest.mark.parametrize("nt,od,id_", SIZES)
@pytest.mark.parametrize("glu", [False, True])
def test_product(qig, nt, od, id_, glu, ytype):
    g = _rng(3, nt, od, id_, glu)
    q, W, sq, sw, b = _operands(g, nt, od * (2 if glu else 1), id_, bias=(nt + od) % 2 == 0)
    ld = _pad(id_, (nt + id_) % 3)
    _say("mm_i8", nt, od, id_, "glu" if glu else "", ytype)
    Wd, qd = _rows(torch.from_numpy(W), ld, 77), _rows(torch.from_numpy(q), _pad(id_, od % 2), -128)
    buf = torch.full((nt + 2, od + 5), 7.0, dtype=TYPES[ytype], device="cuda")
    want, allow = ref.product(q, sq, W, sw, b, glu, ytype)
    for ws in (None, qig.workspace(qd.device)):
        y = buf[1:nt + 1, 2:od + 2]
        y.fill_(float("nan"))
        qig.mm_i8(Wd, _dev(sw), qd, _dev(sq), bias=_dev(b), glu=glu, y=y, ws=ws)
        _check(y, want, allow, (nt, od, id_, ws is not None))
        y.fill_(7.0)
        assert (buf == 7.0).all(), "written outside y"


def test_product_largest_sums(qig):
    """The longest sum of the largest products: 131071 * 2^14 < 2^31."""
    n = 131071
    q = torch.full((2, _pad(n)), -128, dtype=torch.int8, device="cuda")[:, :n]
    W = torch.full((3, _pad(n)), -128, dtype=torch.int8, device="cuda")[:, :n]
    one = torch.ones(3, device="cuda")
    for ws in (None, qig.workspace(q.device)):
        y = qig.mm_i8(W, one, q, one[:2], ws=ws)
        # one rounding of the sum to fp32, two products with 1
        assert (y.cpu().double() == float(np.float32(n * 16384))).all()


@pytest.mark.parametrize("nt,od,id_", [(1, 3584, 3584), (16, 512, 3584), (64, 256, 4096), (100, 700, 2000),
                                       (512, 512, 3584)])
def test_product_same_bits_with_workspace(qig, nt, od, id_):
    g = _rng(4, nt, od)
    q, W, sq, sw, b = _operands(g, nt, od, id_, True)
    a = [_dev(v) for v in (W, sw, q, sq)]
    ws = qig.new_workspace(a[0].device)
    y0 = qig.mm_i8(*a, bias=_dev(b))
    for _ in range(3):
        y1 = qig.mm_i8(*a, bias=_dev(b), ws=ws)
        assert torch.equal(y0, y1)
    assert int(torch.count_nonzero(ws[-16384:])) == 0, "arrival counters not returned to zero"


def test_product_of_quantized_matrices(qig):
    """A linear layer from floating weights and activations, end to end."""
    g = _rng(5)
    x, w = g.standard_normal((50, 777)).astype(np.float32), g.standard_normal((90, 777)).astype(np.float32)
    W, sw = qig.quantize_i8(_dev(w))
    q, sq = qig.quantize_i8(_dev(x))
    y = qig.mm_i8(W, sw, q, sq)
    rW, rsw = ref.quantize(w)
    rq, rsq = ref.quantize(x)
    want, allow = ref.product(rq, rsq, rW, rsw, None, False, "float32")
    _check(y, want, allow, "linear")
    # and near the unquantized product: each operand is off by half a step at most
    full = x.astype(np.float64) @ w.astype(np.float64).T
    off = np.abs(x).sum(1)[:, None] * rsw / 2 + np.abs(w).sum(1) * rsq[:, None] / 2 + 777 * rsq[:, None] * rsw / 4
    assert (np.abs(_np(y) - full) <= off + allow).all()


# --- routing ------------------------------------------------------------------------------------------------

ROUTES = [dict(ne=8, k=2), dict(ne=1, k=1), dict(ne=5, k=5), dict(ne=64, k=6), dict(ne=65, k=8), dict(ne=100, k=32),
          dict(ne=128, k=8, score="sigmoid", bias=True), dict(ne=256, k=8, score="sigmoid", bias=True, groups=8,
                                                              topk_groups=4, group_top=2),
          dict(ne=160, k=6, groups=8, topk_groups=3), dict(ne=160, k=6, groups=8, topk_groups=3, group_top=2),
          dict(ne=512, k=10, score="sigmoid", scale=2.5), dict(ne=48, k=4, bias=True, renorm=False),
          dict(ne=64, k=1, groups=64, topk_groups=5, score="sigmoid", group_top=2), dict(ne=300, k=7, renorm=False),
          dict(ne=16, k=4, groups=4, topk_groups=1, bias=True)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_routing(qig, case, kind):
    c = dict(ROUTES[case])
    ne, k, bias = c.pop("ne"), c.pop("k"), c.pop("bias", False)
    g = _rng(6, case)
    l = torch.from_numpy(g.standard_normal((203, ne)).astype(np.float32) * 2).to(TYPES[kind])
    l[::5] = torch.round(l[::5])                                  # many equal logits
    l[3, :] = 0.25
    l[10:20][torch.from_numpy(g.random((10, ne)) < 0.6)] = float("-inf")
    l[21, :] = float("-inf")
    l[22, :] = float("nan")
    l[23, 0] = float("inf")
    l[24, :] = float("-inf")
    l[24, ne // 2] = -60000.0
    b = (g.standard_normal(ne) * 0.2).astype(np.float32) if bias else None
    _say("route_experts", kind, ne, k, c)
    view = _rows(l, ne + 3)
    ids, w = qig.route_experts(view, k, bias=_dev(b), **c)
    rids, rw = ref.route(l.float().numpy(), k, bias=b, **c)
    got = ids.cpu().numpy()
    # In 64 bits two unequal candidates are never nearer than their rounding here; equal logits are equal scores.
    assert np.array_equal(got, rids), np.argwhere(got != rids)[:4]
    # one rounding to fp32 after 64-bit arithmetic; below 2^-126 a step is 2^-149
    assert (np.abs(w.cpu().numpy() - rw) <= np.abs(rw) * 2.0 ** -23 + 2.0 ** -149).all()


def test_routing_far_logits_keep_their_order(qig):
    """Softmax scores that underflow still choose by logit."""
    l = torch.tensor([[0.0, -2000.0, -1000.0, -3000.0]])
    ids, w = qig.route_experts(l.cuda(), 3)
    assert ids.tolist() == [[0, 2, 1]] and w.tolist() == [[1, 0, 0]]


# --- plan ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("nrows,ne", [(0, 4), (1, 1), (1, 300), (63, 2), (64, 8), (65, 64), (1000, 7), (1024, 512),
                                      (1025, 16), (5000, 200), (15780, 64), (70001, 511), (150000, 3)])
@pytest.mark.parametrize("spread", ["even", "one", "dropped"])
def test_plan(qig, nrows, ne, spread):
    g = _rng(7, nrows, ne)
    ids = g.integers(0, ne, nrows).astype(np.int32)
    if spread == "one":
        ids[:] = ne - 1
    elif spread == "dropped":
        ids[g.random(nrows) < 0.3] = -1
        ids[g.random(nrows) < 0.1] = ne + 5
    _say("plan_experts", nrows, ne, spread)
    out = torch.full((ne + 2 + nrows + 3,), 123, dtype=torch.int32, device="cuda")
    qig.plan_experts(_dev(ids), ne, out=out)
    got = out.cpu().numpy()
    assert np.array_equal(got[:-3], ref.plan(ids, ne))
    assert (got[-3:] == 123).all()


# --- the experts' products ----------------------------------------------------------------------------------

def _experts_case(g, nt, k, ne, od, id_, glu, per_row, spread):
    rows = od * (2 if glu else 1)
    q, W, sq, sw, b = _operands(g, nt * (k if per_row else 1), ne * rows, id_, True)
    ids = np.stack([g.permutation(ne)[:k] for _ in range(nt)]).astype(np.int32).reshape(-1)
    if spread == "one":
        ids[:] = min(1, ne - 1)
    elif spread == "dropped":
        ids[g.random(nt * k) < 0.4] = -1
    elif spread == "none":
        ids[:] = -1
    return q, W, sq, sw, b, ids


EXPERTS = [(1, 1, 1, 1, 1), (1, 2, 4, 33, 17), (3, 2, 5, 64, 128), (4, 6, 64, 130, 200), (16, 4, 8, 100, 256),
           (40, 2, 3, 257, 127), (64, 8, 16, 96, 384), (130, 3, 4, 140, 129), (300, 4, 70, 48, 64), (700, 2, 2, 65, 130),
           (257, 1, 300, 20, 48)]


@pytest.mark.parametrize("nt,k,ne,od,id_", EXPERTS)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("spread", ["even", "one", "dropped", "none"])
def test_experts_product(qig, nt, k, ne, od, id_, glu, spread):
    per_row = (nt + od) % 2 == 0
    ytype = list(TYPES)[(nt + ne + glu) % 3]
    g = _rng(8, nt, ne, od, glu)
    q, W, sq, sw, b, ids = _experts_case(g, nt, k, ne, od, id_, glu, per_row, spread)
    rows = od * (2 if glu else 1)
    _say("mm_i8_experts", nt, k, ne, od, id_, "glu" if glu else "", spread, ytype, "per row" if per_row else "shared")
    Wd = _rows(torch.from_numpy(W), _pad(id_, 1), 99)
    Wd = torch.as_strided(Wd, (ne, rows, id_), (rows * Wd.stride(0), Wd.stride(0), 1), 0)
    qd = _rows(torch.from_numpy(q), _pad(id_), -1)
    plan = qig.plan_experts(_dev(ids), ne)
    n = nt * k
    buf = torch.full((n + 2, od + 5), 7.0, dtype=TYPES[ytype], device="cuda")
    y = buf[1:n + 1, 2:od + 2]
    y.fill_(float("nan"))
    qig.mm_i8_experts(Wd, _dev(sw).view(ne, rows), qd, _dev(sq), plan, n, bias=_dev(b).view(ne, rows), glu=glu, y=y)
    got = _np(y)
    assert np.isfinite(got).all()
    for e in range(-1, ne):
        mine = np.flatnonzero(ids == e)
        if not len(mine):
            continue
        if e < 0:
            assert (got[mine] == 0).all()
            continue
        src = mine if per_row else mine // k
        want, allow = ref.product(q[src], sq[src], W[e * rows:(e + 1) * rows], sw[e * rows:(e + 1) * rows],
                                  b[e * rows:(e + 1) * rows], glu, ytype)
        _check(y[torch.from_numpy(mine).cuda()], want, allow, ("expert", e))
    y.fill_(7.0)
    assert (buf == 7.0).all(), "written outside y"


# --- combine ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("th", list(TYPES))
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("nt,k,od,off", [(1, 1, 1, 0), (3, 2, 7, 1), (5, 6, 64, 0), (2, 8, 1000, 3), (9, 4, 3584, 0),
                                         (40, 3, 257, 2)])
def test_combine(qig, nt, k, od, off, th, ty):
    g = _rng(9, nt, k, od)
    h = torch.from_numpy(g.standard_normal((nt * k, od + off)).astype(np.float32)).to(TYPES[th])
    w = g.random((nt, k)).astype(np.float32)
    _say("combine_experts", nt, k, od, off, th, ty)
    buf = torch.full((nt + 2, od + off + 1), 7.0, dtype=TYPES[ty], device="cuda")
    y = buf[1:nt + 1, off:od + off]
    qig.combine_experts(h.cuda()[:, off:], _dev(w), y=y)
    p = w[:, :, None].astype(np.float64) * h[:, off:].double().numpy().reshape(nt, k, od)
    want = p.sum(1)
    # k products and k sums in fp32, then one rounding
    d = 2 * k * 2.0 ** -24 * np.abs(p).sum(1)
    _check(y, want, d + ref.EPS[ty] * (np.abs(want) + d) + ref.FLOOR[ty], (nt, k, od))
    y.fill_(7.0)
    assert (buf == 7.0).all(), "written outside y"


# --- together -----------------------------------------------------------------------------------------------

def _layer_weights(qig, g, ne, id_, ff):
    up = torch.from_numpy(g.standard_normal((ne * 2 * ff, id_)).astype(np.float32)).cuda() / id_ ** 0.5
    dn = torch.from_numpy(g.standard_normal((ne * id_, ff)).astype(np.float32)).cuda() / ff ** 0.5
    (W1, s1), (W2, s2) = qig.quantize_i8(up), qig.quantize_i8(dn)
    shape = lambda W, r: torch.as_strided(W, (ne, r, W.shape[1]), (r * W.stride(0), W.stride(0), 1))  # noqa: E731
    return shape(W1, 2 * ff), s1.view(ne, -1), shape(W2, id_), s2.view(ne, -1)


def _layer(qig, logits, x, weights, k):
    W1, s1, W2, s2 = weights
    ids, rw = qig.route_experts(logits, k)
    plan = qig.plan_experts(ids, W1.shape[0])
    n = ids.numel()
    q, sq = qig.quantize_i8(x)
    h = qig.mm_i8_experts(W1, s1, q, sq, plan, n, glu=True)
    q, sq = qig.quantize_i8(h)
    h = qig.mm_i8_experts(W2, s2, q, sq, plan, n)
    return ids, qig.combine_experts(h, rw)


@pytest.mark.parametrize("nt,ne,k,id_,ff", [(1, 8, 2, 256, 96), (37, 16, 4, 200, 130), (150, 6, 3, 128, 64)])
def test_experts_layer(qig, nt, ne, k, id_, ff):
    """Routing, plan, both products and the weighted sum as a layer calls
    them, the hidden values taken from the kernels for the second
    quantization (a value at a border may round either way)."""
    g = _rng(10, nt, ne)
    weights = _layer_weights(qig, g, ne, id_, ff)
    x = g.standard_normal((nt, id_)).astype(np.float32)
    l = g.standard_normal((nt, ne)).astype(np.float32)
    l[nt // 2, : ne - 1] = -np.inf                     # one expert left: slots without one
    _say("experts layer", nt, ne, k, id_, ff)
    ids, y = _layer(qig, _dev(l), _dev(x), weights, k)
    rids, rw = ref.route(l, k)
    assert np.array_equal(ids.cpu().numpy(), rids)
    W1, s1, W2, s2 = [w.cpu().numpy() for w in weights]
    q, sq = ref.quantize(x)
    plan = qig.plan_experts(ids, ne)
    dq, dsq = qig.quantize_i8(_dev(x))
    h = qig.mm_i8_experts(weights[0], weights[1], dq, dsq, plan, nt * k, glu=True).cpu().numpy()
    hq, hs = ref.quantize(h)
    want, allow = np.zeros((nt, id_)), np.zeros((nt, id_))
    for t in range(nt):
        for s in range(k):
            e, r = rids[t, s], t * k + s
            if e < 0:
                assert (h[r] == 0).all()
                continue
            hw, ha = ref.product(q[t:t + 1], sq[t:t + 1], W1[e], s1[e], None, True, "float32")
            assert (np.abs(h[r] - hw[0]) <= ha[0]).all()
            o, oa = ref.product(hq[r:r + 1], hs[r:r + 1], W2[e], s2[e], None, False, "float32")
            want[t] += rw[t, s] * o[0]
            # the weight's rounding, and the product's and the sum's in fp32
            allow[t] += rw[t, s] * oa[0] + (2 * k + 1) * 2.0 ** -24 * np.abs(rw[t, s] * o[0])
    _check(y, want, allow + 2.0 ** -140, "layer")


def test_layer_on_other_streams_and_in_graphs(qig):
    """The layer on a stream of its own and replayed from two graphs that
    share their weights, each replay against the eager result."""
    g = _rng(11)
    weights = _layer_weights(qig, g, 8, 256, 128)
    xs = [torch.from_numpy(g.standard_normal((33, 256)).astype(np.float32)).cuda() for _ in range(3)]
    ls = [torch.from_numpy(g.standard_normal((33, 8)).astype(np.float32)).cuda() for _ in range(3)]
    eager = [_layer(qig, l, x, weights, 2)[1].clone() for l, x in zip(ls, xs)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [_layer(qig, l, x, weights, 2)[1] for l, x in zip(ls, xs)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, got))
    W, sw = weights[0][0], weights[1][0]
    lin = [qig.mm_i8(W, sw, *qig.quantize_i8(x)) for x in xs]
    graphs = []
    for _ in range(2):
        x, l, ws = torch.zeros_like(xs[0]), torch.zeros_like(ls[0]), qig.new_workspace(xs[0].device)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y = _layer(qig, l, x, weights, 2)[1]
            z = qig.mm_i8(W, sw, *qig.quantize_i8(x), ws=ws)
        graphs.append((gr, x, l, y, z))
    for i in range(6):
        gr, x, l, y, z = graphs[i % 2]
        x.copy_(xs[i % 3])
        l.copy_(ls[i % 3])
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i % 3]) and torch.equal(z, lin[i % 3]), i
        assert torch.equal(_layer(qig, ls[0], xs[0], weights, 2)[1], eager[0])


def test_nothing_to_do(qig):
    """No tokens, no outputs, no rows."""
    z = lambda *n, t=torch.float32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    i8 = torch.int8
    q, s = qig.quantize_i8(z(0, 40))
    assert q.shape == (0, 40) and s.shape == (0,)
    assert qig.mm_i8(z(8, 32, t=i8), z(8), z(0, 32, t=i8), z(0)).shape == (0, 8)
    assert qig.mm_i8(z(0, 32, t=i8), z(0), z(3, 32, t=i8), z(3)).shape == (3, 0)
    ids, w = qig.route_experts(z(0, 8), 2)
    assert ids.shape == w.shape == (0, 2)
    plan = qig.plan_experts(ids, 8)
    assert plan.tolist() == [0] * 10
    assert qig.mm_i8_experts(z(8, 4, 32, t=i8), z(8, 4), z(0, 32, t=i8), z(0), plan, 0).shape == (0, 4)
    assert qig.combine_experts(z(0, 16), z(0, 2)).shape == (0, 16)
    torch.cuda.synchronize()


def test_given_stream_and_two_streams_at_once(qig):
    """Calls on two streams, each with a workspace of its own, on shapes that
    split their sums, interleaved on the host."""
    g = _rng(12)
    q, W, sq, sw, _ = _operands(g, 100, 300, 4000, False)
    a = [_dev(v) for v in (W, sw, q, sq)]
    y0 = qig.mm_i8(*a)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [qig.new_workspace(a[0].device) for _ in range(2)]
    torch.cuda.synchronize()
    ys = [[torch.empty_like(y0) for _ in range(5)] for _ in range(2)]
    for i in range(5):
        for s in range(2):
            qig.mm_i8(*a, y=ys[s][i], ws=ws[s], stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(y, y0) for r in ys for y in r)


def test_default_workspace_in_captures_and_on_a_given_stream(qig):
    """Split products whose workspace is the default one of a stream that has
    none yet: two captures on one stream, the second replayed first, and a
    stream passed to the call while another is current."""
    g = _rng(13)
    nt, od, id_ = 70, 200, 8192
    q, W, sq, sw, _ = _operands(g, nt, od, id_, False)
    a = (_dev(W), _dev(sw), _dev(q), _dev(sq))
    want = qig.mm_i8(*a)
    outs = [torch.zeros_like(want) for _ in range(3)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = []
    for y in outs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            for _ in range(2):
                qig.mm_i8(*a, y=y, ws=qig.workspace(a[0].device))
        graphs.append(gr)
    for i in (1, 0, 1, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want), i
    t = torch.cuda.Stream()
    qig.mm_i8(*a, y=outs[2], ws=qig.workspace(a[0].device, t), stream=t)
    t.synchronize()
    assert torch.equal(outs[2], want)
    assert qig.workspace(a[0].device, t).data_ptr() == qig.workspace(a[0].device, t).data_ptr()


def _same_up_to_rounding(got, want, what):
    """fp32 results of two kernels on the same integer sum, |bias| <= 4: the
    conversion and two products round by 2^-24 of |y| + |bias| each, the
    addition by 2^-24 of |y|, in both, so they differ by at most 8 (|y| +
    |bias|) 2^-24."""
    err = ((got.double() - want.double()).abs() / (want.double().abs() + 4.0)).max().item()
    _say(what, err)
    assert err <= 8 * 2.0 ** -24, what


def test_rows_behind_32_bit_offsets(qig):
    """Tensors whose last rows lie more than 2^31 elements or 2^32 bytes behind
    their first, each checked against the same rows alone."""
    torch.manual_seed(5)
    nt, id_ = 270000, 16384                                   # x: 8.8 GB, q: 4.4 GB
    x = torch.empty((nt, id_), dtype=torch.bfloat16, device="cuda").normal_()
    q, s = qig.quantize_i8(x)
    for lo, hi in ((0, 40), (131000, 131100), (nt - 40, nt)):
        q1, s1 = qig.quantize_i8(x[lo:hi].clone())
        assert torch.equal(q1, q[lo:hi]) and torch.equal(s1, s[lo:hi]), lo
    del x
    W, sw = qig.quantize_i8(torch.randn(24, id_, device="cuda"))
    bias = torch.randn(24, device="cuda").clamp_(-4, 4)
    y = torch.zeros((nt, 8192), device="cuda")[:, :24]        # 2.2e9 elements, 8.8 GB
    qig.mm_i8(W, sw, q, s, bias=bias, y=y)
    for lo, hi in ((0, 8), (131000, 131070), (262130, 262160), (nt - 9, nt)):
        _same_up_to_rounding(y[lo:hi], qig.mm_i8(W, sw, q[lo:hi], s[lo:hi], bias=bias), f"rows {lo}")
    del y
    # experts: the same rows, every fourth of a second expert, the last dropped
    W2, sw2 = torch.stack([W, W.flip(0)]), torch.stack([sw, sw.flip(0)])
    ids = (torch.arange(nt, device="cuda", dtype=torch.int32) % 4 == 3).int()
    ids[-1] = -1
    plan = qig.plan_experts(ids, 2)
    y = torch.zeros((nt, 8192), device="cuda")[:, :24]
    y[-1] = 7
    qig.mm_i8_experts(W2, sw2, q, s, plan, nt, y=y)
    for lo, hi in ((0, 8), (131000, 131070), (262130, 262160), (nt - 9, nt)):
        r = torch.arange(lo, hi, device="cuda")
        for e in range(2):
            rows = r[ids[lo:hi] == e]
            _same_up_to_rounding(y[rows], qig.mm_i8(W2[e], sw2[e], q[rows], s[rows]), f"expert {e}, rows {lo}")
    assert int(torch.count_nonzero(y[-1])) == 0
    # h [2 * 135000][8192] of the same storage
    w = torch.rand(nt // 2, 2, device="cuda")
    z = qig.combine_experts(y, w)
    for lo, hi in ((0, 8), (131065, 131080), (nt // 2 - 8, nt // 2)):
        assert torch.equal(z[lo:hi], qig.combine_experts(y[2 * lo:2 * hi].clone(), w[lo:hi])), lo
    del y, q
    # weights: 2 x 1100 x 16384 of 130 experts, 4.7 GB
    W = torch.randint(-127, 128, (130, 2200, id_), dtype=torch.int8, device="cuda")
    sw = torch.rand(130, 2200, device="cuda") * 1e-4
    q, s = qig.quantize_i8(torch.randn(60, id_, device="cuda"))
    for n in (3, 60):
        ids = torch.tensor([129, 119, 0] * 20, dtype=torch.int32, device="cuda")[:n]
        y = qig.mm_i8_experts(W, sw, q[:n], s[:n], qig.plan_experts(ids, 130), n, glu=True)
        for e in (129, 119, 0):
            rows = (ids == e).nonzero()[:, 0]
            a, b = (qig.mm_i8(W[e, i:i + 1100], sw[e, i:i + 1100], q[rows], s[rows]).double() for i in (0, 1100))
            want = a * torch.sigmoid(a) * b
            # in 2^-24 of |a b|: a and b are 4 roundings off in either kernel
            # (times silu's slope, 1.1, for a), the activation 8 + 3 |a|
            err = ((y[rows].double() - want).abs() / ((26 + 3 * a.abs()) * (a * b).abs() + 2.0 ** -100)).max().item()
            _say("expert", e, err)
            assert err <= 2.0 ** -24, e
    del W, y
    # logits [8.5e6][512] fp16, 8.7 GB
    nt = 8500000
    l = torch.empty((nt, 512), dtype=torch.float16, device="cuda").normal_()
    ids, w = qig.route_experts(l, 4)
    for lo, hi in ((0, 40), (4194290, 4194320), (8388590, 8388620), (nt - 9, nt)):
        i1, w1 = qig.route_experts(l[lo:hi].clone(), 4)
        assert torch.equal(i1, ids[lo:hi]) and torch.equal(w1, w[lo:hi]), lo


def test_routing_group_sums_beyond_fp32(qig):
    """Two largest biases whose sum no fp32 holds: the groups are told apart in
    64 bits all the same, and infinite biases tie towards the lower group."""
    logits = torch.zeros(1, 8, device="cuda")
    route = lambda b, **kw: qig.route_experts(logits, 2, score="sigmoid", groups=4, topk_groups=1, group_top=2,  # noqa: E731
                                              bias=torch.tensor(b, device="cuda"), **kw)[0].tolist()
    assert route([3e38, 2e38, 3e38, 3.1e38, 3e38, 1.5e38, 0, 0]) == [[3, 2]]
    assert route([-3.3e38, -3e38, -3.2e38, -3e38, -3.3e38, -3.1e38, -3.3e38, -3.2e38]) == [[3, 2]]
    inf = float("inf")
    assert route([0, 0, inf, 1, inf, 5, inf, inf]) == [[2, 3]]
    assert route([-inf, -inf, -inf, -inf, -inf, 0, -inf, -inf]) == [[5, -1]]
    assert route([-inf, -inf, float("nan"), -3e38, -inf, -inf, -3.3e38, -3.3e38]) == [[3, -1]]


# (tokens, k, experts, weight rows): few rows of many experts (weights beyond the register kernel's range), few tiles,
# more than the CUs, and enough for 128- and 256-row tiles
EXPERT_TILES = {"few rows": (12, 6, 64, 0), "few tiles": (40, 2, 3, 406), "tiles": (100, 4, 8, 3350),
                "128 rows": (80, 4, 16, 6430), "256 rows": (210, 4, 8, 7010)}


@pytest.mark.parametrize("id_", [17, 129, 256, 300, 512, 600, 1000])
@pytest.mark.parametrize("form", list(EXPERT_TILES))
def test_experts_product_every_tile(qig, form, id_):
    """Each tile form through one to eight steps, whole and with a tail, on
    ragged rows and outputs: the first, middle and last experts' outputs."""
    nt, k, ne, rows = EXPERT_TILES[form]
    rows = rows or (25400000 // (ne * id_) + 7) // 2 * 2
    glu = (id_ + ne) % 2 == 0
    od = rows // 2 if glu else rows
    torch.manual_seed(id_)
    _say("mm_i8_experts", form, id_, rows, "glu" if glu else "")
    W = torch.randint(-128, 128, (ne, rows, _pad(id_)), dtype=torch.int8, device="cuda")[:, :, :id_]
    sw = torch.rand(ne, rows, device="cuda") * 0.02 + 1e-4
    q = torch.randint(-127, 128, (nt, _pad(id_)), dtype=torch.int8, device="cuda")[:, :id_]
    sq = (torch.rand(nt, device="cuda") * 0.02 + 1e-3) / max(1.0, id_ ** 0.5 / 4)
    bias = torch.randn(ne, rows, device="cuda")
    ids = torch.rand(nt, ne, device="cuda").argsort(1)[:, :k].int().contiguous()
    ids[0] = ne - 1                                        # the same expert in every slot
    ids[1, 0] = -1
    y = torch.full((nt * k, od + 3), 7.0, device="cuda")
    qig.mm_i8_experts(W, sw, q, sq, qig.plan_experts(ids, ne), nt * k, bias=bias, glu=glu, y=y[:, :od])
    assert bool((y[:, od:] == 7.0).all()) and bool((y[k, :od] == 0).all())
    flat = ids.flatten().cpu().numpy()
    for e in (0, ne // 2, ne - 1):
        mine = np.flatnonzero(flat == e)
        want, allow = ref.product(q.cpu().numpy()[mine // k], sq.cpu().numpy()[mine // k], W[e].cpu().numpy(),
                                  sw[e].cpu().numpy(), bias[e].cpu().numpy(), glu, "float32")
        _check(y[torch.from_numpy(mine).cuda()][:, :od], want, allow, (form, e))


@pytest.mark.parametrize("id_", [17, 129, 256, 300, 512, 600, 1000])
@pytest.mark.parametrize("nt,rows", [(600, 4002), (1530, 7930), (2630, 4790)])
def test_product_every_tile(qig, nt, rows, id_):
    """The larger tiles through one to eight steps, whole and with a tail, on
    ragged tokens and outputs: sampled tokens' outputs."""
    glu = id_ % 3 == 0
    od = rows // 2 if glu else rows
    torch.manual_seed(id_)
    _say("mm_i8", nt, rows, id_, "glu" if glu else "")
    W = torch.randint(-128, 128, (rows, _pad(id_)), dtype=torch.int8, device="cuda")[:, :id_]
    sw = torch.rand(rows, device="cuda") * 0.02 + 1e-4
    q = torch.randint(-127, 128, (nt, _pad(id_)), dtype=torch.int8, device="cuda")[:, :id_]
    sq = (torch.rand(nt, device="cuda") * 0.02 + 1e-3) / max(1.0, id_ ** 0.5 / 4)
    bias = torch.randn(rows, device="cuda")
    y = torch.full((nt + 1, od + 3), 7.0, device="cuda")
    qig.mm_i8(W, sw, q, sq, bias=bias, glu=glu, y=y[:nt, :od])
    assert bool((y[:, od:] == 7.0).all()) and bool((y[nt] == 7.0).all())
    t = torch.cat([torch.arange(3), torch.randint(0, nt, (40,)), torch.arange(nt - 20, nt)])
    want, allow = ref.product(q.cpu().numpy()[t], sq.cpu().numpy()[t], W.cpu().numpy(), sw.cpu().numpy(),
                              bias.cpu().numpy(), glu, "float32")
    _check(y[t.cuda()][:, :od], want, allow, (nt, rows, id_))


@pytest.mark.parametrize("nt", [1, 2, 4, 5])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("ne,k,groups,keep", [(511, 16, 7, 3), (510, 17, 30, 5), (96, 24, 32, 20), (441, 32, 63, 40),
                                              (33, 31, 11, 11), (512, 2, 2, 1)])
def test_routing_many_chosen_and_odd_groups(qig, nt, score, ne, k, groups, keep):
    """16 and more experts a token, groups of odd sizes, and token counts on
    both sides of a workgroup's, with and without renormalisation."""
    g = _rng(14, nt, ne)
    l = g.standard_normal((nt, ne)).astype(np.float32) * 2
    l[nt - 1, g.random(ne) < 0.5] = -np.inf
    b = (g.standard_normal(ne) * 0.2).astype(np.float32)
    for renorm in (True, False):
        kw = dict(score=score, groups=groups, topk_groups=keep, group_top=2, renorm=renorm, scale=1.5)
        ids, w = qig.route_experts(_dev(l), k, bias=_dev(b), **kw)
        rids, rw = ref.route(l, k, bias=b, **kw)
        assert np.array_equal(ids.cpu().numpy(), rids)
        assert (np.abs(w.cpu().numpy() - rw) <= np.abs(rw) * 2.0 ** -23 + 2.0 ** -149).all()
