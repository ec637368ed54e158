"""The 4-bit cache: its bytes, what it stands for, and the attention over it."""
import math
import random

import numpy as np
import pytest
import torch

import attend_ref as ref
import quant_integer_gemm_amd as qig

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def rows(n, heads, d, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, d), generator=g) * spread
    x *= torch.rand((1, heads, d), generator=g) * 2 + 0.2
    return (x + torch.randn((1, heads, d), generator=g)).to(dtype).cuda()


class Cache:
    """Sequences in scattered pages; room: entries of the table beyond the needed ones."""

    def __init__(self, lens, heads, d, page, seed=1, room=1, spare=3):
        rng = random.Random(seed)
        counts = [-(-n // page) for n in lens]
        order = list(range(sum(counts) + spare))
        rng.shuffle(order)
        width = max(counts + [0]) + room
        t = [[order.pop() for _ in range(c)] + [-1] * (width - c) for c in counts]
        self.pages = qig.new_kv4(sum(counts) + spare, heads, d, page)
        self.pages.fill_(0xff)                     # NaN scales wherever nothing is written
        self.tables = ints(t) if t else torch.empty((0, width), dtype=torch.int32, device="cuda")
        self.lengths, self.d = ints(lens), d

    def write(self, k, v, starts=None, lengths=None):
        qig.write_kv4(k, v, self.pages, self.tables, self.lengths if lengths is None else lengths, starts)

    def read(self, n, starts=None, **kw):
        return qig.read_kv4(self.pages, self.tables, self.lengths, self.d, starts, n, **kw)


def filled(lens, heads, d, page, dtype=F32, seed=1, **kw):
    c = Cache(lens, heads, d, page, seed, **kw)
    c.k, c.v = rows(sum(lens), heads, d, dtype, seed + 10), rows(sum(lens), heads, d, dtype, seed + 11)
    c.write(c.k, c.v, ints(starts_of(lens)))
    return c


# --- write and read --------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_bytes(d, dtype):
    """A whole page, byte for byte by the layout's text."""
    c = filled([64], 2, d, 64, dtype, spare=0)
    got = c.pages.cpu().numpy()[0]
    kc, ks, km = ref.quantize4(c.k.float().cpu().numpy())
    vc, vs, vm = ref.quantize4(c.v.float().cpu().numpy())
    for head in range(2):
        for b in range(2):
            t = slice(32 * b, 32 * b + 32)
            want = ref.block_bytes(kc[t, head], ks[t, head], km[t, head], vc[t, head], vs[t, head], vm[t, head])
            assert np.array_equal(got[head, b * 40 * d:(b + 1) * 40 * d], want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d,page,heads,lens", [
    (64, 32, 1, [1]), (128, 64, 4, [5, 0, 64, 65, 130, 31]), (256, 128, 3, [200, 1]), (64, 96, 8, [97, 300]),
])
def test_values(d, page, heads, lens, dtype):
    c = filled(lens, heads, d, page, dtype, 3)
    k, v = c.read(sum(lens), ints(starts_of(lens)))
    assert np.array_equal(k.cpu().numpy(), ref.stands_for(c.k.float().cpu().numpy()))
    assert np.array_equal(v.cpu().numpy(), ref.stands_for(c.v.float().cpu().numpy()))
    for t in (BF16, F16):
        k2, v2 = c.read(sum(lens), ints(starts_of(lens)), dtype=t)
        assert torch.equal(k2, k.to(t)) and torch.equal(v2, v.to(t))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_borders(dtype):
    """Values halfway between two codes, equal ones, zeros of both signs, the smallest and
    the largest, and ranges far from zero."""
    d = 64
    g = torch.Generator().manual_seed(1)
    x = torch.zeros((12, 1, d), dtype=torch.float64)
    x[0] = torch.randint(0, 31, (1, d), generator=g) / 2.0           # ties: m = 0, s = 1
    x[0, 0, ::32], x[0, 0, 1::32] = 0, 15
    x[1] = torch.randint(-15, 16, (1, d), generator=g) / 2.0
    x[2] = 3.0
    x[3] = 1.0 + 2.0 ** -7
    x[4, 0, ::2] = -0.0
    x[5] = torch.randn((1, d), generator=g) * 1e-6
    x[6] = torch.randn((1, d), generator=g) * 1e4
    x[7] = 500 + torch.rand((1, d), generator=g)
    x[8] = -500 - torch.rand((1, d), generator=g)
    x[9, 0, 5] = 1.0
    x[10] = torch.randn((1, d), generator=g) * (1e-39 if dtype != F16 else 1e-7)
    x[11] = torch.randn((1, d), generator=g) * (1e37 if dtype != F16 else 2e4)
    x = x.to(dtype)
    c = Cache([12], 1, d, 32)
    c.write(x.cuda(), x.cuda(), ints([0, 12]))
    k, v = c.read(12, ints([0, 12]))
    want = ref.stands_for(x.float().numpy())
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)
    _, s, _ = ref.quantize4(x.float().numpy())
    off = np.abs(want.astype(np.float64) - x.double().numpy()).reshape(12, 1, 2, 32)
    assert (off <= s[..., None] * 0.5 + np.abs(want.reshape(off.shape)) * 2.0 ** -24).all()


@pytest.mark.parametrize("ratio", [0, 4, 12])
def test_values_next_to_borders(ratio):
    """fp32 values a few steps to either side of where a code begins, next to minima up to
    2^ratio times the scale."""
    n, d = 600, 128
    g = torch.Generator().manual_seed(ratio)
    s = (torch.rand((n, 1, d // 32, 1), generator=g) + 0.5).bfloat16().float()
    m = ((torch.rand((n, 1, d // 32, 1), generator=g) - 0.5) * 2.0 ** ratio).bfloat16().float()
    code = torch.randint(0, 15, (n, 1, d // 32, 32), generator=g)
    x = (m.double() + (code.double() + 0.5) * s.double()).float()
    x = (x.view(torch.int32) + torch.randint(-3, 4, x.shape, generator=g, dtype=torch.int32)).view(torch.float32)
    x[..., :1], x[..., 1:2] = m, (m.double() + 15 * s.double()).float()
    x = x.reshape(n, 1, d)
    c = Cache([n], 1, d, 32)
    c.write(x.cuda(), -x.cuda(), ints([0, n]))
    k, v = c.read(n, ints([0, n]))
    # a few steps below 0 in bits is NaN: those groups stand for NaN, the others for numbers
    for got, of in ((k, x), (v, -x)):
        of = of.numpy().reshape(n, -1, 32)
        nan = np.isnan(of).any(2)
        want = ref.stands_for(np.where(nan[..., None], 0, of).reshape(n, 1, d)).reshape(of.shape)
        want[nan] = math.nan
        assert np.array_equal(got.cpu().numpy().reshape(of.shape), want, equal_nan=True) and nan.mean() < 0.01


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(bad):
    """A group that holds one stands for NaN, the others for what they are."""
    x = rows(3, 1, 128, F32, 1)
    x[1, 0, 40] = bad
    c = Cache([3], 1, 128, 32)
    c.write(x, x, ints([0, 3]))
    k, v = c.read(3, ints([0, 3]))
    for t in (k, v):
        nan = t.isnan().cpu()
        assert nan[1, 0, 32:64].all() and nan.sum() == 32


def test_token_by_token():
    """One token a call (without starts) leaves the same bytes as all at once."""
    n, heads, d = 70, 2, 128
    whole = filled([n, n], heads, d, 32)
    c = Cache([n, n], heads, d, 32)
    for i in range(n):
        c.write(whole.k[[i, n + i]], whole.v[[i, n + i]], None, ints([i + 1, i + 1]))
    assert torch.equal(c.pages, whole.pages)


def test_write_leaves_the_rest():
    """Only the new tokens' bytes change, and nothing where no page is."""
    c = filled([50, 40], 2, 64, 32)
    before = c.read(90, ints([0, 50, 90]))
    pages = c.pages.clone()
    none = c.tables.clone()
    none[:, :] = -1
    none[0, 0] = c.pages.shape[0]
    qig.write_kv4(c.k, c.v, c.pages, none, c.lengths, ints([0, 50, 90]))
    qig.write_kv4(c.k[:9], c.v[:9], c.pages, c.tables, ints([0, 4]), ints([0, 4, 9]))   # 4 before the start, and one
    qig.write_kv4(c.k[:5], c.v[:5], c.pages, c.tables, ints([5000, -3]), ints([0, 2, 5]))
    qig.write_kv4(c.k[:0], c.v[:0], c.pages, c.tables, c.lengths, ints([0, 0, 0]))
    k, v = c.read(90, ints([0, 50, 90]))
    changed = torch.zeros(90, dtype=torch.bool)
    changed[50:54] = True
    assert torch.equal(k[~changed], before[0][~changed]) and torch.equal(v[~changed], before[1][~changed])
    assert np.array_equal(k[50:54].cpu().numpy(), ref.stands_for(c.k[5:9].cpu().numpy()))
    qig.write_kv4(c.k[50:], c.v[50:], c.pages, c.tables, ints([50, 40]), ints([0, 0, 40]))
    assert torch.equal(c.pages, pages)


def test_read_nowhere():
    c = filled([40], 2, 64, 32)
    k = torch.full((46, 2, 64), 9.0, device="cuda")
    v = k.clone()
    t = c.tables.clone()
    t[0, 1] = -1
    qig.read_kv4(c.pages, t, ints([36]), 64, ints([2, 44]), k=k, v=v)
    assert (k[:2] == 9).all() and (k[44:] == 9).all()
    assert (k[2:8] == 0).all() and (v[2:8] == 0).all()               # positions -6 .. -1
    assert np.array_equal(k[8:40].cpu().numpy(), ref.stands_for(c.k[:32].cpu().numpy()))
    assert (k[40:44] == 0).all()                                     # the second page


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strides(dtype):
    """Parts of one product's output at odd addresses; layers in one pool."""
    n, heads, d = 45, 3, 64
    flat = torch.randn((n, 2 * heads * d + 5), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()[:, 3:]
    k, v = (flat[:, i * heads * d:(i + 1) * heads * d].unflatten(1, (heads, d)) for i in (0, 1))
    plain = Cache([n], heads, d, 32)
    plain.write(k.contiguous(), v.contiguous(), ints([0, n]))
    pool = torch.full((plain.pages.shape[0], 2) + plain.pages.shape[1:], 0xff, dtype=torch.uint8, device="cuda")
    st = ints([0, n])
    qig.write_kv4(k, v, pool[:, 1], plain.tables, plain.lengths, st)
    assert torch.equal(pool[:, 1], plain.pages) and (pool[:, 0] == 0xff).all()
    both = torch.zeros((n, 2 * heads * d + 5), dtype=dtype, device="cuda")[:, 1:]
    k2, v2 = (both[:, i * heads * d:(i + 1) * heads * d].unflatten(1, (heads, d)) for i in (0, 1))
    qig.read_kv4(pool[:, 1], plain.tables, plain.lengths, d, st, k=k2, v=v2)
    want = plain.read(n, st, dtype=dtype)
    assert torch.equal(k2, want[0]) and torch.equal(v2, want[1])
    wide = torch.full((1, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :plain.tables.shape[1]] = plain.tables
    q = rows(n, 6, d, dtype, 5)
    ys = [qig.attend_kv4(q, p, t, plain.lengths, st) for p in (plain.pages, pool[:, 1])
          for t in (plain.tables, wide[:, :plain.tables.shape[1]], wide)]
    assert all(torch.equal(y, ys[0]) for y in ys)


# --- attention ------------------------------------------------------------------------------------------------------

def attend(c, lens, new, hq, dtype, out=None, scale=None, ws=None, seed=5, spread=1.0, tables=None, seen=None):
    """Runs and checks; the queries are the last new[s] tokens."""
    heads, d, dev = c.pages.shape[1], c.d, "cuda"
    q = rows(sum(new), hq, d, dtype, seed, spread)
    st = None if new == [1] * len(lens) else ints(starts_of(new))
    y = qig.attend_kv4(q, c.pages, c.tables if tables is None else tables, c.lengths, st, scale=scale, dtype=out, ws=ws)
    torch.cuda.synchronize()
    scale = 1 / math.sqrt(d) if scale is None else scale
    kq, vq = ref.quantize4(c.k.float().cpu().numpy()), ref.quantize4(c.v.float().cpu().numpy())
    ks, vs = (torch.from_numpy(ref.values4(*x)) for x in (kq, vq))
    # sizes of the terms: |m| + s c
    size = lambda x: torch.from_numpy(ref.values4(x[0], x[1], np.abs(x[2])))  # noqa: E731
    ka, va = size(kq), size(vq)
    at = a = 0
    for s, (n, total) in enumerate(zip(new, lens)):
        qs = q[a:a + n]
        pos = [total - n + i for i in range(n)]
        sl = slice(at, at + total)
        see = None if seen is None else seen[s]
        w, _, _ = ref.attention(qs, ks[sl], vs[sl], n, pos, scale, see)
        amax = torch.einsum("ihd,jhd->ihj", qs.double().abs().cpu(),
                            ka[sl].double().repeat_interleave(hq // heads, 1)) * scale
        amax = amax.amax(2, keepdim=True) if total else torch.zeros((n, hq, 1), dtype=torch.float64)
        # p is the same as in the result: the sizes' average with it
        _, mag, _ = ref.attention(qs, ks[sl], va[sl], n, pos, scale, see)
        smax = float(vq[1][sl].max()) if total else 0.0
        amp = float(qs.double().abs().max() * ka[sl].abs().sum(-1).max()) * scale if total and n else 0.0
        allow = ref.kv4_allowance(qs, mag, amax, amp, d, total, dtype, y.dtype, smax)(w)
        ref.check(y[a:a + n], w, allow, f"sequence {s}: {n} of {total}")
        at, a = at + total, a + n
    return q, y


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths(d, dtype, ws):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 300, 1000]
    c = filled(lens, 2, d, 64, dtype)
    attend(c, lens, [1] * len(lens), 8, dtype, ws=qig.new_workspace("cuda") if ws else None)


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype,out", [(F32, BF16), (F32, F16), (BF16, F32), (BF16, F16), (F16, F32), (F16, BF16)])
def test_output_types(dtype, out, ws):
    lens = [70, 700]
    attend(filled(lens, 2, 128, 32), lens, [1, 1], 4, dtype, out, ws=qig.new_workspace("cuda") if ws else None)


@pytest.mark.parametrize("heads,hq", [(1, 1), (1, 7), (4, 28), (8, 8), (2, 32), (1, 40), (3, 48)])
def test_head_layouts(heads, hq):
    lens = [33, 257]
    attend(filled(lens, heads, 64, 32), lens, [1, 1], hq, BF16, ws=qig.new_workspace("cuda"))


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens,new", [
    ([50, 200, 7], [5, 5, 5]), ([40, 64, 0, 33], [40, 3, 0, 0]), ([300, 300], [1, 130]), ([0, 0], [0, 0]),
    ([3, 0, 40], [10, 4, 41]),                      # more queries than tokens: the first ones see nothing
    ([64, 96, 128], [33, 32, 31]),
])
def test_several_queries(lens, new, dtype, ws):
    c = filled(lens, 2, 64, 32)
    attend(c, lens, new, 6, dtype, ws=qig.new_workspace("cuda") if ws else None)


@pytest.mark.parametrize("page", [32, 64, 96, 256])
def test_pages_and_long_sequences(page):
    """One long sequence among short ones, in pages of all sizes: rows of many pieces."""
    lens = [20000, 3, 50, 4097, 1, 800]
    attend(filled(lens, 2, 128, page), lens, [1] * 6, 14, BF16, ws=qig.new_workspace("cuda"))


def test_many_sequences():
    """More sequences than a workgroup sums at once."""
    rng = random.Random(1)
    lens = [rng.choice([0, 1, 2, 5, 33, 70]) for _ in range(700)]
    c = filled(lens, 1, 64, 32)
    attend(c, lens, [1] * 700, 2, BF16, ws=qig.new_workspace("cuda"))
    attend(c, lens, [rng.randint(0, 2) for _ in range(700)], 2, BF16)


def test_no_sequences():
    c = Cache([], 2, 64, 32)
    y = qig.attend_kv4(rows(1, 4, 64, BF16, 1)[:0], c.pages, c.tables, c.lengths)
    assert y.shape == (0, 4, 64)


@pytest.mark.parametrize("ws", [False, True])
def test_table_too_short_and_missing_pages(ws):
    """Pages that the table does not have are left out; so are tokens beyond it."""
    lens = [200, 200]
    c = filled(lens, 2, 64, 32, room=0)
    t = c.tables.clone()
    t[0, 2], t[1, 0], t[1, 4] = -1, c.pages.shape[0], -7
    seen = [torch.ones(200, dtype=torch.bool) for _ in range(2)]
    seen[0][64:96] = False
    seen[1][0:32] = seen[1][128:160] = False
    w = qig.new_workspace("cuda") if ws else None
    attend(c, lens, [1, 1], 4, BF16, ws=w, tables=t, seen=seen)
    attend(c, lens, [40, 9], 4, F32, ws=w, tables=t, seen=seen)
    short = [torch.arange(200) < 160, torch.arange(200) < 160]
    attend(c, lens, [1, 1], 4, BF16, ws=w, tables=c.tables[:, :5], seen=short)
    none = torch.zeros_like(t) - 1
    y = qig.attend_kv4(rows(2, 4, 64, BF16, 1), c.pages, none, c.lengths, ws=w)
    assert (y == 0).all()
    y = qig.attend_kv4(rows(2, 4, 64, BF16, 1), c.pages, none[:, :0], c.lengths, ws=w)
    assert (y == 0).all()


@pytest.mark.parametrize("scale,spread", [(1e-3, 1.0), (1.0, 1.0), (2.0, 3.0), (None, 1e-4), (None, 1e3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scales(scale, spread, dtype):
    lens = [300, 45]
    attend(filled(lens, 2, 64, 32), lens, [1, 3], 4, dtype, scale=scale, spread=spread, ws=qig.new_workspace("cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_values_of_different_sizes(dtype):
    """Values whose scales grow, shrink and differ between groups by 2^40: the reference
    of a group moves, and others' stay exact."""
    lens = [400]
    c = Cache(lens, 1, 128, 32)
    c.k, c.v = rows(400, 1, 128, F32, 1), rows(400, 1, 128, F32, 2)
    e = torch.linspace(-20, 20, 400, device="cuda")
    c.v[:, :, :32] *= torch.exp2(e)[:, None, None]
    c.v[:, :, 32:64] *= torch.exp2(-e)[:, None, None]
    c.v[:, :, 64:96] *= 2.0 ** -60
    c.v[:, :, 96:] *= 2.0 ** 60 if dtype != F16 else 1.0
    c.write(c.k, c.v, ints([0, 400]))
    q = rows(1, 4, 128, dtype, 3)
    y = qig.attend_kv4(q, c.pages, c.tables, c.lengths, dtype=F32)
    kq, vq = ref.quantize4(c.k.cpu().numpy()), ref.quantize4(c.v.cpu().numpy())
    ks, vs = (torch.from_numpy(ref.values4(*x)) for x in (kq, vq))
    w, _, _ = ref.attention(q, ks, vs, 1, [399], 1 / math.sqrt(128))
    for g in range(4):
        sl = slice(32 * g, 32 * g + 32)
        _, mag, _ = ref.attention(q, ks, torch.from_numpy(ref.values4(vq[0], vq[1], np.abs(vq[2]))), 1, [399],
                                  1 / math.sqrt(128))
        amax = (q.double().abs().cpu() @ torch.from_numpy(np.abs(ks.numpy())).double()[:, 0].T).amax(2, keepdim=True)
        allow = ref.kv4_allowance(q, mag[..., sl], amax / math.sqrt(128), float(amax.max()), 128, 400, dtype, F32,
                                  float(vq[1][:, 0, g].max()))(w[..., sl])
        ref.check(y[..., sl], w[..., sl], allow, f"group {g}")


@pytest.mark.parametrize("ws", [False, True])
def test_unseen_tokens_hold_anything(ws):
    """NaN in tokens that come after a query, and in what the pages hold behind the end."""
    lens = [100, 64]
    c = filled(lens, 2, 64, 32)
    q = rows(9, 4, 64, BF16, 1)
    st, w = ints([0, 6, 9]), qig.new_workspace("cuda") if ws else None
    clean = qig.attend_kv4(q, c.pages, c.tables, c.lengths, st, ws=w)
    k, v = c.k.clone(), c.v.clone()
    k[97:100], v[97:100] = math.nan, math.inf       # the first sequence's last three
    c.write(k, v, ints(starts_of(lens)))
    y = qig.attend_kv4(q, c.pages, c.tables, c.lengths, st, ws=w)
    assert torch.equal(y[:3], clean[:3]) and torch.equal(y[6:], clean[6:]) and y[3:6].isnan().all()


def test_rows_outside_are_left():
    lens = [100, 64]
    c = filled(lens, 2, 64, 32)
    q = rows(12, 4, 64, F16, 1)
    y = torch.full((12, 4, 70), 7.0, dtype=F16, device="cuda")
    qig.attend_kv4(q, c.pages, c.tables, c.lengths, ints([2, 5, 10]), y=y[:, :, 3:67])
    assert (y[:2] == 7).all() and (y[10:] == 7).all() and (y[:, :, :3] == 7).all() and (y[:, :, 67:] == 7).all()
    want = qig.attend_kv4(q[2:10], c.pages, c.tables, c.lengths, ints([0, 3, 8]))
    assert torch.equal(y[2:10, :, 3:67], want)


def test_wrong_starts_and_lengths_stay_inside():
    c = filled([100, 64], 2, 64, 32)
    q, pages = rows(40, 4, 64, BF16, 1), c.pages.clone()
    y = torch.full((60, 4, 64), 5.0, dtype=BF16, device="cuda")
    w = qig.new_workspace("cuda")
    for st in ([0, 500, 20], [-40, 30, 20], [50, 10, -3], [0, 2147483647, -2147483648]):
        for lengths in ([100, 64], [2147483647, -2147483648], [0, 1 << 20]):
            qig.attend_kv4(q, c.pages, c.tables, ints(lengths), ints(st), y=y[10:50], ws=w)
            qig.attend_kv4(q, c.pages, c.tables, ints(lengths), ints(st), y=y[10:50])
            qig.read_kv4(c.pages, c.tables, ints(lengths), 64, ints(st), k=y[10:50, :2], v=y[10:50, 2:])
            torch.cuda.synchronize()
            assert (y[:10] == 5).all() and (y[50:] == 5).all()
    assert torch.equal(c.pages, pages)


@pytest.mark.parametrize("nseq", [63, 2001])
def test_starts_that_ask_for_too_much(nseq):
    """Starts up and down, so that the sequences together ask for more than 2^32 blocks (none
    of which has a page): nothing outside is touched, and the workspace serves the next call."""
    c = filled([300, 64], 1, 64, 32)
    w = qig.new_workspace("cuda")
    q, two = rows(2000, 16, 64, BF16, 1), rows(2, 16, 64, BF16, 2)
    want = qig.attend_kv4(two, c.pages, c.tables, c.lengths, ws=w)
    width = 16384 if nseq > 100 else 1 << 18
    # the longest list that is counted: nt * 16 / 16 + nseq rows by width + 1 blocks
    assert (2000 + nseq) * (width + 1) < 2 ** 31 < 2 ** 32 < (nseq // 2) * 2000 * width
    tables = torch.full((nseq, width), -1, dtype=torch.int32, device="cuda")
    y = torch.full((2020, 16, 64), 5.0, dtype=BF16, device="cuda")
    st = ints([0 if i % 2 == 0 else 2000 for i in range(nseq + 1)])
    qig.attend_kv4(q, c.pages, tables, ints([width * 32] * nseq), st, y=y[10:2010], ws=w)
    torch.cuda.synchronize()
    assert (y[:10] == 5).all() and (y[2010:] == 5).all()
    assert torch.equal(qig.attend_kv4(two, c.pages, c.tables, c.lengths, ws=w), want)
    many = qig.attend_kv4(rows(64, 16, 64, BF16, 3), c.pages, c.tables[:1].expand(64, -1).contiguous(),
                          ints([300] * 64), ws=w)
    assert not many.isnan().any() and (many != 0).any(2).all()


def test_the_same_on_every_call():
    lens = [5000, 70, 900]
    c = filled(lens, 2, 128, 64)
    q, w = rows(3, 14, 128, BF16, 1), qig.new_workspace("cuda")
    y = qig.attend_kv4(q, c.pages, c.tables, c.lengths, ws=w)
    for _ in range(5):
        assert torch.equal(qig.attend_kv4(q, c.pages, c.tables, c.lengths, ws=w), y)
    assert int(torch.count_nonzero(w[-16384:])) == 0    # the products' counters are not touched


def test_far_pages():
    """Pages behind 2^32 bytes."""
    heads, d, page, n = 8, 128, 64, 100
    c = filled([n], heads, d, page, spare=0)
    far = (1 << 32) // (c.pages.shape[1] * c.pages.shape[2]) + 100
    pages = torch.empty((far + 2,) + c.pages.shape[1:], dtype=torch.uint8, device="cuda")
    t = c.tables.clone()
    t[0, 0], t[0, 1] = far + 1, far
    st = ints([0, n])
    qig.write_kv4(c.k, c.v, pages, t, c.lengths, st)
    assert torch.equal(pages[far + 1], c.pages[c.tables[0, 0]])
    q = rows(1, 8, d, BF16, 1)
    assert torch.equal(qig.attend_kv4(q, pages, t, c.lengths), qig.attend_kv4(q, c.pages, c.tables, c.lengths))
    assert torch.equal(qig.read_kv4(pages, t, c.lengths, d, st, n)[1], c.read(n, st)[1])
