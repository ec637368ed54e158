"""Routing where scores are nearer than fp32 can tell apart."""
import numpy as np
import pytest

import int8_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


# c = p + bias; `near` logits differ by a few steps of fp32, nearer than the 32-bit choice can tell
NEAR = [dict(score="sigmoid"), dict(score="sigmoid", bias=True), dict(score="softmax", bias=True)]


@pytest.mark.parametrize("kind", range(len(NEAR)))
@pytest.mark.parametrize("ne,k", [(8, 3), (64, 6), (200, 8), (300, 31), (512, 1)])
@pytest.mark.parametrize("many", [2, 3, 30])
def test_near_values(qig, kind, ne, k, many):
    """`many` unequal values next to each other, placed among the chosen,
    across the border of the chosen, and right behind it; the other experts
    far above and below."""
    c = dict(NEAR[kind])
    g = np.random.Generator(np.random.PCG64([20263, kind, ne, k, many]))
    many = min(many, ne - 1)
    nt = 61
    l = np.empty((nt, ne), np.float32)
    b = np.zeros(ne, np.float32) if c.pop("bias", False) else None
    for t in range(nt):
        above = max(0, min(k + 1 - t % (many + 2), ne - many))   # clearly larger ones
        x = np.concatenate([3 + 0.05 * np.arange(above), 1 + np.float32(2.0 ** -23) * g.permutation(40)[:many],
                            -3 - 0.01 * np.arange(ne - many - above)])
        l[t] = g.permutation(x.astype(np.float32))
    if b is not None:
        # differences of the biases near those of the scores, the same for all tokens
        b = (g.integers(0, 8, ne) * 2.0 ** -30).astype(np.float32)
    ids, w = qig.route_experts(_dev(l), k, bias=_dev(b), **c)
    rids, rw = ref.route(l, k, bias=b, **c)
    got = ids.cpu().numpy()
    assert np.array_equal(got, rids), np.argwhere(got != rids)[:4]
    assert (np.abs(w.cpu().numpy() - rw) <= np.abs(rw) * 2.0 ** -23).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("ne,groups,keep,k", [(16, 4, 2, 4), (64, 8, 4, 6), (252, 7, 3, 8), (512, 64, 32, 10)])
def test_near_groups(qig, score, top, ne, groups, keep, k):
    """Groups whose scores are nearer than fp32 can tell: two at the border of
    those that stay, then all of them."""
    g = np.random.Generator(np.random.PCG64([20264, ne, top, len(score)]))
    size, nt = ne // groups, 64
    l = (-4 - g.random((nt, ne))).astype(np.float32)
    for t in range(nt):
        order = g.permutation(groups)
        for i, gr in enumerate(order):
            near = t % 2 == 1 or keep - 1 <= i <= keep
            base = 1.0 if near else (2.0 + 0.1 * i if i < keep else 0.5 - 0.001 * i)
            for e in g.permutation(size)[:2]:
                # multiples of 8 steps: the sums of two differ by far more than 64 bits round
                l[t, gr * size + e] = np.float32(base) + np.float32(2.0 ** -20) * g.integers(0, 20)
    b = (g.standard_normal(ne) * 2.0 ** -32).astype(np.float32) if score == "softmax" else None
    kw = dict(score=score, groups=groups, topk_groups=keep, group_top=top)
    ids, w = qig.route_experts(_dev(l), k, bias=_dev(b), **kw)
    rids, rw = ref.route(l, k, bias=b, **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, rids), np.argwhere(got != rids)[:4]
    assert (np.abs(w.cpu().numpy() - rw) <= np.abs(rw) * 2.0 ** -23).all()
