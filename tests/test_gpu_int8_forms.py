"""Every kernel form of the int8 products, the form asserted: each through one
to eight steps of 128 bytes, whole and with a tail, with last tiles of every
height, gated and not, in every output type; and sums split into two, three and
four shares."""
import numpy as np
import pytest

import int8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
IDS = [17, 129, 256, 300, 512, 600, 1000]


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


def _kind(i):
    """Gated or not, and the output type: all six in turn."""
    return i % 2 == 1, list(TYPES)[i // 2 % 3]


def _pad(n):
    return (n + 15) // 16 * 16


def _operands(shape, id_, nt):
    """Weights of `shape` rows, activations, scales and biases; outputs of
    order one."""
    W = torch.randint(-128, 128, (*shape, _pad(id_)), dtype=torch.int8, device="cuda")[..., :id_]
    sw = torch.rand(shape, device="cuda") * 0.02 + 1e-4
    q = torch.randint(-127, 128, (nt, _pad(id_)), dtype=torch.int8, device="cuda")[:, :id_]
    sq = (torch.rand(nt, device="cuda") * 0.02 + 1e-3) / max(1.0, id_ ** 0.5 / 4)
    return W, sw, q, sq, torch.randn(shape, device="cuda")


def _np(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _check(y, want, allow, what):
    got = _np(y).astype(np.float64)
    assert np.isfinite(got).all(), what
    worst = float((np.abs(got - want) / allow).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"


# (form, tokens, weight rows): the last tile's tokens are 37, 101, 165 or 229
DENSE = [(6421, 600, 4002), (6421, 700, 3002), (19221, 1381, 4402), (19221, 1061, 5860), (19221, 2469, 2458),
         (25621, 1573, 6346), (25621, 1381, 7318), (25621, 1189, 8290), (25621, 997, 9748)]


@pytest.mark.parametrize("step", range(len(IDS)))
@pytest.mark.parametrize("shape", range(len(DENSE)))
def test_dense_forms(qig, shape, step):
    form, nt, rows = DENSE[shape]
    id_ = IDS[step]
    glu, kind = _kind(shape + step)
    od = rows // 2 if glu else rows
    assert qig.load().mm_i8_form(0, od, id_, nt, int(glu), 0) == form
    torch.manual_seed(100 * shape + step)
    print("mm_i8", form, nt, od, id_, "glu" if glu else "", kind, flush=True)
    W, sw, q, sq, bias = _operands((rows,), id_, nt)
    y = torch.full((nt + 1, od + 3), 7.0, dtype=TYPES[kind], device="cuda")
    qig.mm_i8(W, sw, q, sq, bias=bias, glu=glu, y=y[:nt, :od])
    assert bool((y[:, od:] == 7.0).all()) and bool((y[nt] == 7.0).all())
    tall = form // 100
    last = nt // tall * tall   # the last tile's first token
    t = torch.cat([torch.arange(3), torch.randint(0, nt, (30,)), torch.randint(last, nt, (20,)), torch.arange(nt - 20, nt)])
    want, allow = ref.product(_np(q)[t], _np(sq)[t], _np(W), _np(sw), _np(bias), glu, kind)
    _check(y[t.cuda()][:, :od], want, allow, (form, nt, rows, id_))


# form: (tokens, k, experts, weight rows, 0: as many as leave the few-token kernel's range)
EXPERTS = [(3241, 12, 6, 64, 0), (6441, 40, 2, 3, 406), (6421, 100, 4, 8, 3350), (12821, 80, 4, 16, 6430),
           (25621, 210, 4, 8, 7010)]


@pytest.mark.parametrize("step", range(len(IDS)))
@pytest.mark.parametrize("shape", range(len(EXPERTS)))
def test_experts_forms(qig, shape, step):
    form, nt, k, ne, rows = EXPERTS[shape]
    id_ = IDS[step]
    rows = rows or (25400000 // (ne * id_) + 7) // 2 * 2
    glu, kind = _kind(shape + step)
    od = rows // 2 if glu else rows
    assert qig.load().mm_i8_form(ne, od, id_, nt * k, int(glu), 0) == form
    torch.manual_seed(10000 + 100 * shape + step)
    print("mm_i8_experts", form, nt, k, ne, od, id_, "glu" if glu else "", kind, flush=True)
    W, sw, q, sq, bias = _operands((ne, rows), id_, nt)
    ids = torch.rand(nt, ne, device="cuda").argsort(1)[:, :k].int().contiguous()
    ids[0] = ne - 1                                        # the same expert in every slot
    ids[1, 0] = -1
    y = torch.full((nt * k, od + 3), 7.0, dtype=TYPES[kind], device="cuda")
    qig.mm_i8_experts(W, sw, q, sq, qig.plan_experts(ids, ne), nt * k, bias=bias, glu=glu, y=y[:, :od])
    assert bool((y[:, od:] == 7.0).all()) and bool((y[k, :od] == 0).all())
    flat = _np(ids).ravel()
    used = np.unique(flat[flat >= 0])
    for e in (used[0], used[len(used) // 2], used[-1]):
        mine = np.flatnonzero(flat == e)
        want, allow = ref.product(_np(q)[mine // k], _np(sq)[mine // k], _np(W[e]), _np(sw[e]), _np(bias[e]), glu, kind)
        _check(y[torch.from_numpy(mine).cuda()][:, :od], want, allow, (form, e))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("shares,nt,od,id_", [(2, 70, 200, 4500), (3, 100, 300, 6211), (4, 130, 130, 8211),
                                              (4, 65, 64, 131071)])
def test_split_sums(qig, shares, nt, od, id_, glu, kind):
    """Shares of different numbers of steps, the last with a tail: the same bits
    as whole sums, in a workspace whose slots were used and whose counters are
    zero after each call."""
    form = qig.load().mm_i8_form
    assert form(0, od, id_, nt, int(glu), 1) == 6440 + shares and form(0, od, id_, nt, int(glu), 0) == 6441
    torch.manual_seed(nt + od)
    print("mm_i8 split", shares, nt, od, id_, "glu" if glu else "", kind, flush=True)
    W, sw, q, sq, bias = _operands(((2 if glu else 1) * od,), id_, nt)
    whole = qig.mm_i8(W, sw, q, sq, bias=bias, glu=glu, dtype=TYPES[kind])
    want, allow = ref.product(_np(q), _np(sq), _np(W), _np(sw), _np(bias), glu, kind)
    _check(whole, want, allow, "whole")
    ws = qig.new_workspace("cuda")
    ws.zero_()
    for _ in range(3):
        y = torch.full((nt + 1, od + 3), 7.0, dtype=TYPES[kind], device="cuda")
        qig.mm_i8(W, sw, q, sq, bias=bias, glu=glu, y=y[:nt, :od], ws=ws)
        assert torch.equal(y[:nt, :od], whole)
        assert bool((y[:, od:] == 7.0).all()) and bool((y[nt] == 7.0).all())
        assert int(torch.count_nonzero(ws[-16384:])) == 0, "arrival counters not returned to zero"
    assert int(torch.count_nonzero(ws[:-16384])) > 0, "no sums in the workspace: not split"
