"""The int8 linear layer and the experts' operators without a GPU: argument
checks of the C ABI and of the binding, and the plain forms of the tests
against hand-made cases."""
import ctypes

import numpy as np
import pytest

import int8_ref as ref
import quant_integer_gemm_amd as qig

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)   # 8-byte aligned only
ODD = ctypes.c_void_p(0x10001)


@pytest.mark.parametrize("args,rc", [
    ((P, 0, 4, 100, 100, P, 112, P, None), None),
    ((P, 3, 4, 100, 100, P, 112, P, None), -1),      # type
    ((P, 0, -1, 100, 100, P, 112, P, None), -1),     # nt
    ((P, 0, 4, 0, 100, P, 112, P, None), -1),        # id
    ((P, 0, 4, 100, 99, P, 112, P, None), -1),       # ldx
    ((P, 0, 4, 100, 100, P, 99, P, None), -1),       # ldq
    ((P, 0, 1 << 31, 100, 100, P, 112, P, None), -1),
    ((P, 0, 4, 1 << 31, 1 << 31, P, 1 << 31, P, None), -1),
    ((None, 0, 4, 100, 100, P, 112, P, None), -1),
    ((P, 0, 4, 100, 100, P, 112, None, None), -1),
    ((ODD, 1, 4, 100, 100, P, 112, P, None), -2),
    ((P, 0, 4, 100, 100, P, 112, ODD, None), -2),
    ((P, 0, 0, 100, 100, P, 112, P, None), 0),       # no rows
])
def test_quantize_i8_argument_checks(args, rc):
    if rc is not None:
        assert qig.load().quantize_i8(*args) == rc


def _mm(**kw):
    a = dict(W=P, ldw=112, sw=P, od=8, id=100, q=P, ldq=112, sq=P, nt=4, bias=None, glu=0, y=P, yt=0, ldy=8, ws=None)
    a.update(kw)
    return qig.load().mm_i8(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(nt=-1), -1), (dict(od=-1), -1), (dict(id=0), -1), (dict(id=131072, ldw=1 << 18, ldq=1 << 18), -1),
    (dict(ldw=96), -1), (dict(ldq=96), -1), (dict(ldy=7), -1), (dict(yt=3), -1), (dict(glu=2), -1),
    (dict(ldw=1 << 23), -1), (dict(ldq=1 << 23), -1), (dict(nt=1 << 31), -1), (dict(od=1 << 30, ldy=1 << 30), -1),
    (dict(ldw=104), -2), (dict(ldq=120), -2), (dict(W=MIS), -2), (dict(q=MIS), -2), (dict(sw=ODD), -2),
    (dict(bias=ODD), -2), (dict(y=ODD, yt=1), -2), (dict(ws=MIS), -2), (dict(W=None), -1), (dict(sq=None), -1),
    (dict(y=None), -1), (dict(nt=0), 0), (dict(od=0), 0), (dict(nt=0, W=None, q=None), 0),
])
def test_mm_i8_argument_checks(kw, rc):
    assert _mm(**kw) == rc


def _mme(**kw):
    a = dict(W=P, ldw=112, sw=P, ne=4, od=8, id=100, q=P, ldq=112, sq=P, nrows=6, slots=2, plan=P, bias=None, glu=0,
             y=P, yt=0, ldy=8)
    a.update(kw)
    return qig.load().mm_i8_experts(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(ne=0), -1), (dict(ne=513), -1), (dict(slots=0), -1), (dict(slots=4), -1), (dict(nrows=1 << 29), -1),
    (dict(plan=None), -1), (dict(plan=ODD), -2), (dict(id=131072, ldw=1 << 18, ldq=1 << 18), -1), (dict(ldw=104), -2),
    (dict(nrows=0), 0), (dict(od=0), 0),
])
def test_mm_i8_experts_argument_checks(kw, rc):
    assert _mme(**kw) == rc


def _route(**kw):
    a = dict(l=P, lt=0, nt=4, ne=16, ldl=16, bias=None, score=0, groups=1, keep=1, top=1, k=4, renorm=1, scale=1.0,
             ids=P, w=P)
    a.update(kw)
    return qig.load().route_experts(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(lt=5), -1), (dict(nt=-1), -1), (dict(ne=0, ldl=0), -1), (dict(ne=513, ldl=513), -1), (dict(ldl=15), -1),
    (dict(score=2), -1), (dict(groups=0), -1), (dict(groups=3), -1), (dict(groups=4, keep=5), -1), (dict(keep=0), -1),
    (dict(top=3), -1), (dict(top=0), -1), (dict(k=0), -1), (dict(k=17), -1), (dict(groups=4, keep=1, k=5), -1),
    (dict(ne=64, ldl=64, k=33), -1), (dict(ne=130, ldl=130, groups=65, keep=65), -1),
    (dict(l=None), -1), (dict(ids=None), -1), (dict(l=ODD), -2), (dict(bias=ODD), -2), (dict(w=ODD), -2),
    (dict(nt=0), 0),
])
def test_route_argument_checks(kw, rc):
    assert _route(**kw) == rc


def test_plan_and_combine_argument_checks():
    lib = qig.load()
    assert qig.expert_plan_bytes(100, 8) == 4 * (100 + 10)
    assert qig.expert_plan_bytes(0, 8) == 40
    for bad in ((-1, 8), (1 << 29, 8), (4, 0), (4, 513)):
        assert qig.expert_plan_bytes(*bad) == 0
        assert lib.plan_experts(P, *bad, P, None) == -1
    assert lib.plan_experts(None, 4, 8, P, None) == -1
    assert lib.plan_experts(P, 4, 8, None, None) == -1
    assert lib.plan_experts(ODD, 4, 8, P, None) == -2
    # (h, type, ldh, w, nt, k, od, y, type, ldy)
    assert lib.combine_experts(P, 3, 8, P, 4, 2, 8, P, 0, 8, None) == -1
    assert lib.combine_experts(P, 0, 8, P, 4, 0, 8, P, 0, 8, None) == -1
    assert lib.combine_experts(P, 0, 7, P, 4, 2, 8, P, 0, 8, None) == -1
    assert lib.combine_experts(P, 0, 8, P, 4, 2, 8, P, 0, 7, None) == -1
    assert lib.combine_experts(P, 0, 8, P, 1 << 30, 2, 8, P, 0, 8, None) == -1
    assert lib.combine_experts(P, 0, 8, None, 4, 2, 8, P, 0, 8, None) == -1
    assert lib.combine_experts(ODD, 1, 8, P, 4, 2, 8, P, 0, 8, None) == -2
    assert lib.combine_experts(P, 0, 8, P, 0, 2, 8, P, 0, 8, None) == 0
    assert lib.combine_experts(P, 0, 0, P, 4, 2, 0, P, 0, 0, None) == 0


def _refused(fn, *words):
    with pytest.raises(qig.QigError) as e:
        fn()
    assert all(w in str(e.value) for w in words), str(e.value)


def test_binding_refuses_wrong_tensors():
    f, i8 = torch.float32, torch.int8
    x, W, q = torch.zeros(3, 32), torch.zeros(5, 32, dtype=i8), torch.zeros(3, 32, dtype=i8)
    sw, sq = torch.zeros(5), torch.zeros(3)
    _refused(lambda: qig.quantize_i8(x), "GPU tensor")
    _refused(lambda: qig.quantize_i8(x.double()), "float32")
    _refused(lambda: qig.quantize_i8(x.t()), "unit column stride")
    _refused(lambda: qig.quantize_i8(x, q=torch.zeros(3, 31, dtype=i8)), "q must be [3][32]")
    _refused(lambda: qig.quantize_i8(x, s=torch.zeros(2)), "s must be contiguous")
    _refused(lambda: qig.mm_i8(W, sw, q, sq), "GPU tensor")
    _refused(lambda: qig.mm_i8(W.float(), sw, q, sq), "W must be torch.int8")
    _refused(lambda: qig.mm_i8(W, sw[:4], q, sq), "sw must be")
    _refused(lambda: qig.mm_i8(W, sw, q, sq[:2]), "sq must be")
    _refused(lambda: qig.mm_i8(W, sw, q[:, :16], sq), "16 columns")
    _refused(lambda: qig.mm_i8(W, sw, q, sq, glu=True), "even number")
    _refused(lambda: qig.mm_i8(W, sw, q, sq, bias=torch.zeros(5, dtype=torch.float16)), "bias")
    _refused(lambda: qig.mm_i8(W, sw, q, sq, y=torch.zeros(3, 4)), "y must be [3][5]")
    _refused(lambda: qig.mm_i8(W, sw, q, sq, dtype=torch.float64), "y must be float32")
    _refused(lambda: qig.mm_i8(W, sw, q, sq, y=torch.zeros(3, 5), dtype=torch.float16), "dtype asks")
    _refused(lambda: qig.mm_i8(W, sw, q, sq, ws=torch.zeros(16, dtype=torch.uint8)), "ws holds")
    # rows that end inside a 16-byte unit at the end of the storage
    _refused(lambda: qig.mm_i8(torch.zeros(5, 30, dtype=i8), sw, torch.zeros(3, 30, dtype=i8), sq), "16-byte unit")
    ids = torch.zeros(3, 2, dtype=torch.int32)
    _refused(lambda: qig.route_experts(x, 2), "GPU tensor")
    _refused(lambda: qig.route_experts(x, 2, score="relu"), "score")
    _refused(lambda: qig.route_experts(x, 2, bias=torch.zeros(31)), "bias")
    _refused(lambda: qig.route_experts(x, 2, ids=torch.zeros(3, 3, dtype=torch.int32)), "ids")
    _refused(lambda: qig.plan_experts(ids, 4), "GPU tensor")
    _refused(lambda: qig.plan_experts(ids.long(), 4), "ids must be torch.int32")
    _refused(lambda: qig.plan_experts(ids, 0), "no plan")
    _refused(lambda: qig.plan_experts(ids, 4, out=torch.zeros(11, dtype=torch.int32)), "out must be")
    We, swe, plan = torch.zeros(4, 5, 32, dtype=i8), torch.zeros(4, 5), torch.zeros(12, dtype=torch.int32)
    _refused(lambda: qig.mm_i8_experts(We, swe, q, sq, plan, 6), "GPU tensor")
    _refused(lambda: qig.mm_i8_experts(We, swe, q, sq, plan, 7), "no multiple")
    _refused(lambda: qig.mm_i8_experts(We, swe, q, sq, plan[:-1], 6), "plan is not one")
    _refused(lambda: qig.mm_i8_experts(We[:, :4], swe[:, :4], q, sq, plan, 6), "follow each other")
    _refused(lambda: qig.mm_i8_experts(We[0], swe, q, sq, plan, 6), "W must be [experts]")
    _refused(lambda: qig.combine_experts(torch.zeros(6, 8), torch.zeros(3, 2)), "GPU tensor")
    _refused(lambda: qig.combine_experts(torch.zeros(5, 8), torch.zeros(3, 2)), "h must be [6]")


def test_plain_quantization_on_hand_made_rows():
    q, s = ref.quantize([[127, -127, 0.5, -0.5, 0.49, 1.5]])
    assert s[0] == 1 and q.tolist() == [[127, -127, 1, -1, 0, 2]]
    q, s = ref.quantize([[0, 0]])
    assert s[0] == 0 and q.tolist() == [[0, 0]]


def test_plain_routing_on_hand_made_rows():
    ids, w = ref.route([[0, 1, 1, -np.inf]], 3)
    assert ids.tolist() == [[1, 2, 0]] and abs(w.sum() - 1) < 1e-12
    ids, w = ref.route([[-np.inf, np.nan, -np.inf, 2]], 2)
    assert ids.tolist() == [[3, -1]] and w.tolist() == [[1, 0]]
    # groups of two: {0, 3}, {2, 2.5}; the best single is in the first, the best pair in the second
    l = [[0.0, 3.0, 2.0, 2.5]]
    assert ref.route(l, 2, "sigmoid", groups=2, topk_groups=1, group_top=1)[0].tolist() == [[1, 0]]
    assert ref.route(l, 2, "sigmoid", groups=2, topk_groups=1, group_top=2)[0].tolist() == [[3, 2]]
    assert ref.plan([[2, 0], [-1, 0]], 3).tolist() == [0, 2, 2, 3, 4, 1, 3, 0, 2]
