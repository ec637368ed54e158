"""Routing by softmax scores that underflow."""
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


def _dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _softmax(l, k, groups, keep, top):
    """Softmax without a bias, from the definition in 64 bits: everything by the
    logits, or, with groups ranked by two scores, everything by p."""
    ids = np.full((len(l), k), -1, np.int32)
    for t, x in enumerate(l.astype(np.float64)):
        ok = x > -np.inf
        c = x
        if top == 2:
            c = np.where(ok, np.exp(np.where(ok, x, 0) - x[ok].max()), 0.0) if ok.any() else np.zeros_like(x)
        size = len(x) // groups
        score = []
        for g in range(groups):
            mine = np.sort(c[g * size:(g + 1) * size][ok[g * size:(g + 1) * size]])[::-1][:top]
            score.append(mine.sum() if len(mine) else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-score[g], g))[:keep]
        mine = [e for e in range(len(x)) if ok[e] and e // size in kept]
        mine = sorted(mine, key=lambda e: (-c[e], e))[:k]
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


@pytest.mark.parametrize("top,want", [(1, [0, 1, 3, 2]), (2, [0, 1, 2, 3])])
def test_underflowing_scores_in_groups(qig, top, want):
    """By logit where groups go by one score; by p, where the last two are both
    0, where they go by two."""
    l = torch.tensor([[0.0, -1.0, -3000.0, -1000.0]], device="cuda")
    ids, w = qig.route_experts(l, 4, groups=2, topk_groups=2, group_top=top)
    assert ids.tolist() == [want]
    assert w[0, 2:].tolist() == [0, 0] and abs(w.sum().item() - 1) < 1e-6


@pytest.mark.parametrize("ne,groups,keep,k", [(8, 2, 2, 8), (64, 8, 3, 12), (60, 6, 4, 9), (256, 8, 4, 8), (512, 4, 2, 32)])
@pytest.mark.parametrize("top", [1, 2])
def test_softmax_in_groups_with_underflow(qig, ne, groups, keep, k, top):
    """Logits over a range in which most scores underflow, equal ones among
    them, some masked."""
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
    got, want = ids.cpu().numpy(), _softmax(l, k, groups, keep, top)
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]
