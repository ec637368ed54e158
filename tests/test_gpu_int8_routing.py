"""Routing where values are near: scores closer than fp32 can tell apart, and
softmax scores that underflow."""
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


def _by_logit(l, k, groups, keep, top):
    """Softmax without a bias, from the definition: the groups by the sum of
    their `top` largest p, the experts by their logits, in 64 bits."""
    ids = np.full((len(l), k), -1, np.int32)
    for t, x in enumerate(l.astype(np.float64)):
        ok = x > -np.inf
        p = np.where(ok, np.exp(np.where(ok, x, 0) - x[ok].max()), 0.0) if ok.any() else np.zeros_like(x)
        size = len(x) // groups
        score = []
        for g in range(groups):
            mine = np.sort(p[g * size:(g + 1) * size][ok[g * size:(g + 1) * size]])[::-1][:top]
            score.append(mine.sum() if len(mine) else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-score[g], g))[:keep]
        mine = [e for e in range(len(x)) if ok[e] and e // size in kept]
        mine = sorted(mine, key=lambda e: (-x[e], e))[:k]
        ids[t, :len(mine)] = mine
    return ids


def _clear(x, groups, top):
    """Whether 64 bits settle the groups' order however exp and a sum round
    there: two scores are sums of the same values, or both underflow, or differ
    by more than 2^-45 of the larger; none is near the smallest number."""
    d = x - x.max()
    if ((d > -760) & (d < -700)).any():
        return False
    best = -np.sort(-d.reshape(groups, -1), axis=1)[:, :top]
    best[best < -745] = -np.inf
    s = np.exp(best).sum(1)
    for i in range(groups):
        for j in range(i):
            if not np.array_equal(best[i], best[j]) and abs(s[i] - s[j]) <= 2.0 ** -45 * max(s[i], s[j]):
                return False
    return True


def test_underflowing_scores_in_groups_keep_the_logits_order(qig):
    l = torch.tensor([[0.0, -1.0, -3000.0, -1000.0]], device="cuda")
    ids, w = qig.route_experts(l, 4, groups=2, topk_groups=2, group_top=2)
    assert ids.tolist() == [[0, 1, 3, 2]]
    assert w[0, 2:].tolist() == [0, 0] and abs(w.sum().item() - 1) < 1e-6


@pytest.mark.parametrize("ne,groups,keep,k", [(8, 2, 2, 8), (64, 8, 3, 12), (60, 6, 4, 9), (256, 8, 4, 8), (512, 4, 2, 32)])
@pytest.mark.parametrize("top", [1, 2])
def test_softmax_in_groups_chooses_by_logit(qig, ne, groups, keep, k, top):
    """Logits over a range in which most scores underflow, equal ones among
    them, some masked: the experts of a token's best groups in the order of
    their logits."""
    g = np.random.Generator(np.random.PCG64([20262, ne, top]))
    l = np.empty((97, ne), np.float32)
    for t in range(len(l)):
        while True:
            x = np.round(g.standard_normal(ne) * (5 if t % 3 == 0 else 800)).astype(np.float32)
            if 5 <= t < 9:
                x[g.random(ne) < 0.5] = -np.inf
            if _clear(x.astype(np.float64), groups, top):
                break
        l[t] = x
    ids, _ = qig.route_experts(_dev(l), k, groups=groups, topk_groups=keep, group_top=top)
    got, want = ids.cpu().numpy(), _by_logit(l, k, groups, keep, top)
    if top == 1:   # a group's score is its largest logit, also where p underflows
        for t in range(len(l)):
            size = ne // groups
            best = [l[t, i * size:(i + 1) * size].max() for i in range(groups)]
            kept = sorted(range(groups), key=lambda i: (-best[i], i))[:keep]
            mine = [e for e in range(ne) if l[t, e] > -np.inf and e // size in kept]
            mine = sorted(mine, key=lambda e: (-l[t, e], e))[:k]
            want[t] = mine + [-1] * (k - len(mine))
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]


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
