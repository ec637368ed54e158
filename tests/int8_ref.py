"""Plain 64-bit forms of the int8 linear layer and the experts' operators, on
the CPU, written from the definitions in include/qig.h."""
import numpy as np


def quantize(x):
    """(q int8, s fp32) of fp32 rows; x may hold any finite values."""
    x = np.asarray(x, dtype=np.float32)
    big = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(len(x), np.float32)
    s = (big / np.float32(127)).astype(np.float32)
    d = np.where(s > 0, s, np.float32(1)).astype(np.float64)[:, None]
    a = np.abs(x.astype(np.float64))
    k = np.floor(a / d)
    # exact: (2k + 1) d and 2a are representable in 64 bits
    k = np.where(2 * a >= (2 * k + 1) * d, k + 1, k)
    q = np.where(s[:, None] > 0, np.copysign(np.minimum(k, 127), x), 0)
    return q.astype(np.int8), s


def sums(q, W):
    """int64 sums of products, exact (below 2^53)."""
    return np.rint(q.astype(np.float64) @ W.astype(np.float64).T)


def silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


EPS = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
FLOOR = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -25}


def product(q, sq, W, sw, bias, glu, ytype):
    """(y, allowance): fp64 result and how far a result computed in fp32 and
    rounded once to ytype may be from it.

    v = P * sq * sw + bias takes at most four fp32 roundings (the conversion
    of P, two products, one sum), each of half a step relative to a value no
    larger than |P sq sw| + |bias|.  silu adds exp2 of a rounded argument
    (relative error 2^-24 * 2 |a| * log2(e) * ln 2 plus an ulp), a sum, a
    reciprocal and two products: (8 + 3 |a|) 2^-24 relative; its slope is at
    most 1.1.  Below 2^-126 / the other factor the exponential over- or
    underflows: an absolute 2^-120 covers it."""
    u = 2.0 ** -24
    P = sums(q, W)
    sq = sq.astype(np.float64)[:, None]
    sw = sw.astype(np.float64)
    b = 0.0 if bias is None else bias.astype(np.float64)
    v = P * sq * sw + b
    dv = 5 * u * (np.abs(P * sq * sw) + np.abs(b) + np.zeros_like(v))
    if glu:
        od = W.shape[0] // 2
        a, up = v[:, :od], v[:, od:]
        f = silu(a)
        y = f * up
        d = np.abs(up) * (1.1 * dv[:, :od] + np.abs(f) * (8 + 3 * np.abs(a)) * u) + np.abs(f) * dv[:, od:] \
            + (1 + np.abs(up)) * 2.0 ** -120
        d = d * (1 + 1e-3)   # the products of two of these errors
    else:
        y, d = v, dv
    return y, d + EPS[ytype] * (np.abs(y) + d) + FLOOR[ytype]


def route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """(ids, w) in 64 bits; logits fp32 [nt][ne]."""
    x = np.asarray(logits, dtype=np.float64)
    ok0 = x > -np.inf
    x = np.where(ok0, np.minimum(x, np.finfo(np.float32).max), 0.0)
    nt, ne = x.shape
    ids = np.full((nt, k), -1, np.int32)
    w = np.zeros((nt, k))
    for t in range(nt):
        ok = ok0[t].copy()
        if score == "softmax":
            top = x[t][ok].max() if ok.any() else 0.0
            e = np.where(ok, np.exp(np.minimum(x[t] - top, 0)), 0.0)
            p = e / e.sum() if e.sum() > 0 else e
        else:
            with np.errstate(over="ignore"):
                p = np.where(ok, 1 / (1 + np.exp(-x[t])), 0.0)
        by_logit = score == "softmax" and bias is None and (groups == 1 or group_top == 1)
        c = x[t].copy() if by_logit else p + (0 if bias is None else bias.astype(np.float64))
        ok &= c > -np.inf
        c = np.where(ok, c, -np.inf)
        if groups > 1:
            size = ne // groups
            gs = []
            for g in range(groups):
                best = np.sort(c[g * size:(g + 1) * size])[::-1][:group_top]
                gs.append(best[0] + sum(b for b in best[1:] if b > -np.inf))
            keep = sorted(range(groups), key=lambda g: (-gs[g], g))[:topk_groups]
            for g in range(groups):
                if g not in keep:
                    ok[g * size:(g + 1) * size] = False
        order = sorted(np.flatnonzero(ok), key=lambda e: (-c[e], e))[:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[order]
        total = w[t].sum()
        if renorm:
            w[t] = w[t] / total if total > 0 else 0.0
        w[t] *= scale
    return ids, w


def plan(ids, ne):
    """The plan's words."""
    ids = np.asarray(ids).reshape(-1)
    e = np.where((ids >= 0) & (ids < ne), ids, ne)
    order = np.argsort(e, kind="stable")
    first = np.searchsorted(e[order], np.arange(ne + 1))
    return np.concatenate([first, [len(ids)], order]).astype(np.int32)
