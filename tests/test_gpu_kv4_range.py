"""attend_kv4 where the sizes of the cached values differ widely: a token that a row does
not see, or to which it gives next to no weight, must not take bits from the others."""
import math

import numpy as np
import pytest
import torch

import attend_ref as ref
import quant_integer_gemm_amd as qig
from test_gpu_kv4 import BF16, F16, F32, Cache, ints, rows

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24


def written(k, v, page=32):
    """A cache of one sequence, and what its keys and values stand for."""
    n, heads, d = k.shape
    c = Cache([n], heads, d, page)
    c.write(k.cuda(), v.cuda(), ints([0, n]))
    kq, vq = ref.quantize4(k.numpy()), ref.quantize4(v.numpy())
    return c, torch.from_numpy(ref.values4(*kq)).double(), [torch.from_numpy(x).double() for x in vq]


def formula(q, k, v, pos, ytype):
    """(y, its allowance, that without the scores' part) in 64 bits.  q [n][hq][d], k
    [nk][hkv][d], v: codes, s and m.

    A score is off by what kv4_allowance counts: (d + 3 + d / 16) half steps of fp32 of its
    terms' sizes, 2^-22 of them for queries in two parts (also allowed to the others, which are
    exact) and 2^-39 of the row's largest |q| of 32 channels in each of them; p by that factor, twice (its sum).
    p s is rounded to f16 once for bf16 results (2^-11), else in two parts (2^-22), and is off
    by no less than 2^-23 of the row's largest p s in the group: half of f16's smallest step,
    2^-25, where the largest is at least 1/4.  Codes are at most 15.  For 16-bit results an
    MFMA keeps 17 bits below the largest product: two steps of that a block of 32 tokens and
    wave.  Sums and powers in fp32 as in allowance(): 3 nk + 32 half steps."""
    q, (codes, s, m) = q.double().cpu(), v
    n, hq, d = q.shape
    nk, hkv, _ = k.shape
    per, G, scale = hq // hkv, d // 32, 1 / math.sqrt(d)
    k = k.repeat_interleave(per, 1)
    codes, s, m = (x.repeat_interleave(per, 1) for x in (codes, s, m))
    see = torch.arange(nk)[None] <= torch.as_tensor(pos)[:, None]
    t = (torch.einsum("ihd,jhd->hij", q, k) * scale).masked_fill(~see[None], -math.inf)
    p = torch.softmax(t, 2)
    # products in place of einsum over tokens that have no weight: 0 * 2^100 is 0 in 64 bits
    y = torch.einsum("hij,jhgc->ihgc", p, m[..., None] + s[..., None] * codes).reshape(n, hq, d)
    mag = torch.einsum("hij,jhgc->ihgc", p, m.abs()[..., None] + s[..., None] * codes).reshape(n, hq, d)
    top = torch.stack([(p * s[:, :, g].T[:, None]).amax(2).T for g in range(G)], 2)      # [n][hq][G]
    top = top.repeat_interleave(32, 2)
    seen_k = torch.where(see[None, :, :, None], k.abs().transpose(0, 1)[:, None], torch.zeros(()).double())
    amax = torch.einsum("ihd,hijd->hij", q.abs(), seen_k).amax(2).T[..., None] * scale
    most = q.abs().unflatten(2, (G, 32)).amax(3).transpose(0, 1)                         # [hq][n][G]
    amp = (most[:, :, None] * seen_k.unflatten(3, (G, 32)).sum(4)).sum(3).amax(2).T[..., None] * scale
    score = (d + 3 + d // 16 + 4) * E32 * amax + 2.0 ** -39 * amp
    step = 2.0 ** -11 if ytype == BF16 else 2.0 ** -22
    err = mag * ((3 * nk + 32) * E32 + step) + nk * 15 * 2.0 ** -23 * top
    if ytype != F32:
        err = err + (nk // 32 + 4) * 2 * 15 * 2.0 ** -17 * top
    return y, *((e + ref.EPS[ytype] * (y.abs() + e) + ref.FLOOR[ytype])
                for e in ((err + mag * 2 * score) * 1.0001, err * 1.0001))


def attend(c, q, st, ytype, ws):
    return qig.attend_kv4(q.cuda(), c.pages, c.tables, c.lengths, st, dtype=ytype,
                          ws=qig.new_workspace("cuda") if ws else None)


def check_seen(y, want, allow, ytype, what):
    """Results inside the type's range; where some allowed value lies outside it an infinity is
    a right result, and the others only have to be as large."""
    most = torch.finfo(ytype).max / 2
    assert (y.double().cpu().abs()[want.abs() - allow > most] > most / 2).all()
    big = want.abs() + allow > most
    ref.check(torch.where(big, 0, y.double().cpu()), torch.where(big, 0, want), allow, what)


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,d", [(F32, 128), (BF16, 128), (F16, 64), (BF16, 256)])
@pytest.mark.parametrize("ratio", [9, 12, 24, 40, 100])
def test_a_large_draft_behind_the_query(ratio, qtype, d, ytype, ws):
    """Five drafted tokens, the last one's values 2^ratio times the others': the four queries
    before it do not see it."""
    for n in (7, 100, 333):
        k, v = rows(n, 2, d, F32, 1).cpu(), rows(n, 2, d, F32, 2).cpu()
        v[-1] *= 2.0 ** ratio
        c, ks, vs = written(k, v)
        q = rows(5, 8, d, qtype, 3)
        y = attend(c, q, ints([0, 5]), ytype, ws)
        want, allow, values = formula(q, ks, vs, [n - 5 + i for i in range(5)], ytype)
        check_seen(y, want, allow, ytype, f"{n} tokens")
        ref.check(y[:4], want[:4], allow[:4], f"{n} tokens, the four before")
        # the same scores over values of one size
        v[-1] /= 2.0 ** ratio
        even = attend(written(k, v)[0], q, ints([0, 5]), ytype, ws)
        ref.check(y[:4], even[:4].double().cpu(), 2 * values[:4], f"{n} tokens, the four before against even values")


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,d", [(F32, 64), (BF16, 128), (F16, 256)])
@pytest.mark.parametrize("ratio", [9, 12, 24, 40, 100])
def test_a_large_value_without_weight(ratio, qtype, d, ytype, ws):
    """A token of values 2^ratio times the others' that every row sees, with a weight that
    leaves nothing of it, at the sequence's start, inside it and at its end."""
    for n, at in ((300, 0), (300, 130), (300, 299), (2000, 5)):
        k, v = rows(n, 1, d, F32, 1).cpu(), rows(n, 1, d, F32, 2).cpu()
        q = rows(1, 4, d, F32, 3).cpu()
        q[:] = 1 + q * 0.01
        q = q.to(qtype)
        k[at] = -200 * math.log(2) / math.sqrt(d)      # a score 2^-200 of an even one
        v[at] *= 2.0 ** ratio
        v[at, :, :32] /= 2.0 ** ratio                  # one group has it as large as others
        c, ks, vs = written(k, v)
        y = attend(c, q, None, ytype, ws)
        want, allow, values = formula(q, ks, vs, [n - 1], ytype)
        ref.check(y, want, allow, f"token {at} of {n}")
        v[at] = 0.0                                    # the same scores, and nothing of that token
        even = attend(written(k, v)[0], q, None, ytype, ws)
        ref.check(y, even.double().cpu(), 2 * values, f"token {at} of {n} against even values")


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,d", [(F32, 64), (BF16, 128), (F16, 128), (BF16, 256)])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -30, 2.0 ** -9])
def test_a_small_value_with_the_weight(size, qtype, d, ytype, ws):
    """A token of next to no values takes nearly all of the weight: what the others leave is the
    result, and keeps its bits."""
    for n, at in ((300, 0), (300, 170), (1111, 0)):
        k, v = rows(n, 1, d, F32, 1).cpu() * 0.1, rows(n, 1, d, F32, 2).cpu()
        q = rows(1, 4, d, F32, 3).cpu()
        q[:] = 1 + q * 0.01
        q = q.to(qtype)
        k[at] = 22 * math.log(2) / math.sqrt(d)        # 2^22 times an even one's weight
        v[at] *= size
        c, ks, vs = written(k, v)
        y = attend(c, q, None, ytype, ws)
        want, allow, _ = formula(q, ks, vs, [n - 1], ytype)
        ref.check(y, want, allow, f"token {at} of {n}")


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,d", [(F32, 64), (BF16, 128), (F16, 128), (BF16, 256)])
def test_many_small_values_with_the_weight(qtype, d, ytype, ws):
    """As above, with whole blocks of zeros ahead of the first values."""
    for n, zeros in ((300, 32), (500, 160), (3000, 129)):
        k, v = rows(n, 1, d, F32, 1).cpu() * 0.1, rows(n, 1, d, F32, 2).cpu()
        q = (1 + rows(1, 4, d, F32, 3).cpu() * 0.01).to(qtype)
        k[:zeros] = 22 * math.log(2) / math.sqrt(d)
        v[:zeros] = 0.0
        c, ks, vs = written(k, v)
        y = attend(c, q, None, ytype, ws)
        want, allow, _ = formula(q, ks, vs, [n - 1], ytype)
        ref.check(y, want, allow, f"{zeros} of {n}")


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,d", [(F32, 64), (BF16, 128), (F16, 128), (BF16, 256)])
@pytest.mark.parametrize("step", [3, 5, 7, -7])
def test_scales_in_steps(step, qtype, d, ytype, ws):
    """Scales that rise by 2^step every 128 tokens (four waves' blocks), or every 32, while the
    weights fall as much: every token counts alike."""
    for each in (128, 32):
        n = 6 * each + 7
        e = (torch.arange(n) // each) * step
        k = (-e * math.log(2) / math.sqrt(d))[:, None, None].expand(n, 1, d).contiguous().float()
        v = rows(n, 1, d, F32, 2).cpu() * torch.exp2(e.double()).float()[:, None, None]
        c, ks, vs = written(k, v)
        q = (1 + rows(1, 4, d, F32, 3).cpu() * 0.001).to(qtype)
        y = attend(c, q, None, ytype, ws)
        want, allow, _ = formula(q, ks, vs, [n - 1], ytype)
        check_seen(y, want, allow, ytype, f"{each} tokens a step")


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, BF16])
def test_scales_up_and_down(ytype, ws):
    """Scales that rise and fall by 2^80 along a sequence while the weights do the opposite, so
    that every token counts."""
    n, d = 500, 128
    k, v = torch.zeros((n, 1, d)), rows(n, 1, d, F32, 2).cpu()
    e = torch.cat([torch.linspace(0, 40, n // 2), torch.linspace(40, 0, n - n // 2)]).round()
    k[:] = (e * math.log(2) / math.sqrt(d))[:, None, None]
    v *= torch.exp2(-e - 20)[:, None, None]
    v[:, :, 32:64] *= torch.exp2(e)[:, None, None]     # and a group that only the weights change
    c, ks, vs = written(k, v)
    q = torch.ones((1, 2, d))
    y = attend(c, q, None, ytype, ws)
    want, allow, _ = formula(q, ks, vs, [n - 1], ytype)
    ref.check(y, want, allow)


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,scale", [(F32, None), (BF16, None), (F32, 1.0), (BF16, 1.0), (F32, 1e30), (F16, 1e30)])
def test_steep_scores(qtype, scale, ytype, ws):
    """Queries and scales at the types' upper ends: scores are finite and far apart, one key has all
    of the weight.  Its score is an eighth above the others' at least, which no rounding of a score
    (2^-17 of its terms) makes up, so that the values' part of the allowance is all of it."""
    n, d, at = 300, 64, 77
    k, v = rows(n, 1, d, F32, 1).cpu().clamp(-2, 0.5), rows(n, 1, d, F32, 2).cpu()
    k[at] = 2.0
    q = 1 + rows(1, 4, d, F32, 3).cpu() * 0.001
    # sum of q k scale at most 64 * 2 * 1.03 * this: below 2^127
    q *= 2.0 ** (119 if scale == 1.0 else 122 if scale is None else 14) / (1 if scale is None else 1.03)
    c, ks, vs = written(k, v)
    q = q.to(qtype)
    assert ks[at].sum() * 0.9 > ks.sum(2)[torch.arange(n) != at].max() and q.isfinite().all()
    y = qig.attend_kv4(q.cuda(), c.pages, c.tables, c.lengths, scale=scale, dtype=ytype,
                       ws=qig.new_workspace("cuda") if ws else None)
    want, _, values = formula(q.double() / q.double().abs().max() * 1e4, ks, vs, [n - 1], ytype)   # as steep, for exp
    ref.check(y, want, values)


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("ytype", [F32, F16, BF16])
@pytest.mark.parametrize("qtype,d,ratio", [(F32, 64, 12), (F32, 128, 24), (F32, 256, 60), (BF16, 128, 24), (BF16, 64, 40),
                                           (BF16, 256, 100), (F16, 128, 20), (F16, 64, 26)])
def test_queries_of_different_sizes(qtype, d, ratio, ytype, ws):
    """One group of a query's channels is 2^ratio times the others' and its keys are that much
    smaller (or zeros): the others' part of the scores keeps its bits."""
    for n, zeros in ((200, False), (333, True)):
        k, v = rows(n, 2, d, F32, 1).cpu(), rows(n, 2, d, F32, 2).cpu()
        q = rows(3, 8, d, F32, 3).cpu()
        half = ratio // 2 if qtype == F16 else 0       # both ends of fp16
        q *= 2.0 ** -half
        k *= 2.0 ** half
        q[:, :4, 32:64] *= 2.0 ** ratio
        q[:, 6:, :32] *= 2.0 ** ratio                  # other rows of a tile, another group; two even ones
        k[:, 0, 32:64] *= 0 if zeros else 2.0 ** -ratio
        k[:, 1, :32] *= 0 if zeros else 2.0 ** -ratio
        q = q.to(qtype)
        c, ks, vs = written(k, v)
        y = attend(c, q, ints([0, 3]), ytype, ws)
        want, allow, _ = formula(q, ks, vs, [n - 3, n - 2, n - 1], ytype)
        ref.check(y, want, allow, f"{n} tokens")


def test_minima_far_below_the_rest():
    """What fp64 rounds away of hi - m is not there: hi = 15 and lo = -2^-70 have s = 1, a code's
    border that lies 2^-70 above a value is met by it."""
    x = torch.zeros((2, 1, 64))
    x[:, 0, ::32], x[:, 0, 1::32] = torch.tensor([[15.0], [-15.0]]), torch.tensor([[-2.0 ** -70], [2.0 ** -70]])
    x[:, 0, 2::32], x[:, 0, 3::32] = 2.5, -2.5
    x[0, 0, 3::32] = 7.0
    x[1, 0, 2::32] = -12.5
    codes, s, m = ref.quantize4(x.numpy())
    assert (s == 1).all() and (m[0] == -2.0 ** -70).all() and (codes[0, 0, :, :4] == [15, 0, 3, 7]).all()
    c, ks, (vc, vs, vm) = written(x, x)
    k, v = qig.read_kv4(c.pages, c.tables, c.lengths, 64, ints([0, 2]), 2)
    assert torch.equal(k.cpu().double(), ks) and torch.equal(v, k)


def test_numbers_of_the_oracle():
    """The oracle's softmax against a sum by hand."""
    k, v = torch.zeros((2, 1, 64)), torch.zeros((2, 1, 64))
    k[1] = math.log(3.0) / 8
    v[0], v[1] = 4.0, 8.0
    ks, vs = ref.stands_for(k.numpy()), [torch.from_numpy(x).double() for x in ref.quantize4(v.numpy())]
    y, allow, _ = formula(torch.ones((1, 1, 64)), torch.from_numpy(ks).double(), vs, [1], F32)
    p = math.exp(float(ks[1, 0].sum()) / 8)
    assert np.allclose(y.numpy(), (4 + 8 * p) / (1 + p), rtol=1e-12) and (allow < 1e-3).all()
