"""attend_prompt against its 64-bit form: head layouts, types, lengths from none to
many tiles, prefixes, strides and what stands in places that are not seen."""
import math

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


def make(lens, klens, hq, hkv, d, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda n, h: (torch.randn((n, h, d), generator=g) * spread).to(dtype).cuda()  # noqa: E731
    return r(sum(lens), hq), r(sum(klens), hkv), r(sum(klens), hkv)


def want(q, k, v, lens, klens, causal, scale, dtype, ytype):
    """(y, allowance) over all packed sequences."""
    ys, al = [], []
    d = q.shape[2]
    a = ka = 0
    for n, nk in zip(lens, klens):
        pos = [nk - n + i if causal else nk - 1 for i in range(n)]
        y, mag, amax = ref.attention(q[a:a + n], k[ka:ka + nk], v[ka:ka + nk], n, pos, scale)
        ys.append(y)
        # 16-bit operands: p is rounded to their type
        step = 0.0 if dtype == F32 else ref.EPS[dtype]
        al.append(ref.allowance(y, mag, amax, d, nk, step, ytype))
        if dtype == F16 and nk:   # below f16's normal range p keeps 2^-31 of its reference, which is at most its maximum
            al[-1] = al[-1] + nk * 2.0 ** -31 * v[ka:ka + nk].double().abs().max().item()
        a, ka = a + n, ka + nk
    return torch.cat(ys), torch.cat(al)


def run(lens, klens, hq, hkv, d, dtype, causal, seed=1, scale=None, out=None):
    q, k, v = make(lens, klens, hq, hkv, d, dtype, seed)
    st, kst = ints(starts_of(lens)), ints(starts_of(klens))
    y = qig.attend_prompt(q, k, v, st, None if lens == klens else kst, causal=causal, scale=scale, dtype=out)
    torch.cuda.synchronize()
    w, al = want(q, k, v, lens, klens, causal, 1 / math.sqrt(d) if scale is None else scale, dtype, y.dtype)
    ref.check(y, w, al, f"{lens} {klens} {hq}/{hkv} {d} {dtype} {causal}")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 300, 513])
def test_lengths(n, dtype):
    run([n], [n], 4, 2, 128, dtype, True, n)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("d", [8, 16, 40, 64, 72, 80, 96, 120, 128, 136, 192, 256])
def test_head_sizes(d, dtype):
    run([70, 3, 150], [70, 3, 150], 2, 1, d, dtype, True, d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (28, 4), (8, 8), (6, 2), (64, 8)])
@pytest.mark.parametrize("causal", [True, False])
def test_head_layouts(hq, hkv, causal):
    run([65, 130], [65, 130], hq, hkv, 64, BF16, causal, hq)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,klens", [
    ([0], [0]), ([0, 5, 0, 0, 200, 1], [0, 5, 0, 0, 200, 1]),   # sequences without tokens
    ([1, 1, 1, 1], [1, 40, 300, 513]),                          # one query against many keys
    ([10, 130, 64], [200, 131, 1000]),                          # prefixes
    ([10, 129, 40], [3, 0, 39]),                                # fewer keys than queries: rows that see none
    ([5, 5], [0, 0]),
    ([300, 300, 300, 300], [300, 333, 300, 600]),
])
def test_packed(lens, klens, causal, dtype):
    run(lens, klens, 4, 2, 64, dtype, causal, 7)


@pytest.mark.parametrize("dtype,out", [(F32, BF16), (F32, F16), (BF16, F32), (BF16, F16), (F16, F32), (F16, BF16)])
def test_output_types(dtype, out):
    run([33, 140], [50, 140], 3, 3, 96, dtype, True, 3, out=out)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 3.0])
def test_scales(scale, dtype):
    run([200], [230], 2, 1, 64, dtype, True, 4, scale=scale)


def test_many_sequences():
    """More sequences than a wave asks about at once, and than its rounds' steps divide."""
    lens = [(i * 7) % 5 for i in range(4999)]
    run(lens, lens, 2, 1, 64, BF16, True, 5)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_parts_of_one_product(dtype):
    """q, k and v as parts of one tensor, from odd addresses and with odd steps."""
    nt, hq, hkv, d = 150, 4, 2, 64
    g = torch.Generator().manual_seed(1)
    both = torch.randn((nt, (hq + 2 * hkv) * d + 3), generator=g).to(dtype).cuda()
    flat = both[:, 1:-2]
    q = flat[:, :hq * d].unflatten(1, (hq, d))
    k = flat[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = flat[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    st = ints([0, 40, 150])
    y = qig.attend_prompt(q, k, v, st)
    assert torch.equal(y, qig.attend_prompt(q.contiguous(), k.contiguous(), v.contiguous(), st))
    w, al = want(q, k, v, [40, 110], [40, 110], True, 1 / 8, dtype, dtype)
    ref.check(y, w, al)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_heads_first(dtype):
    """[heads][tokens][d] in memory, for the inputs and a given y; shared keys by a stride of 0."""
    n, hq, d = 77, 4, 64
    q, k, v = make([n], [n], hq, hq, d, dtype, 1)
    first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    st = ints([0, n])
    y = torch.empty((hq, n, d), dtype=dtype, device="cuda").transpose(0, 1)
    out = qig.attend_prompt(first(q), first(k), first(v), st, y=y)
    assert out is y and torch.equal(y, qig.attend_prompt(q, k, v, st))
    one = k[:, :1].expand(n, hq, d)
    assert torch.equal(qig.attend_prompt(q, one, one, st), qig.attend_prompt(q, k[:, :1], k[:, :1], st))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_rows_outside_are_left(dtype):
    q, k, v = make([200], [200], 2, 1, 80, dtype, 1)
    y = torch.full((200, 2, 80), 7.0, dtype=dtype, device="cuda")
    wide = torch.full((200, 2, 90), 7.0, dtype=dtype, device="cuda")
    qig.attend_prompt(q, k, v, ints([5, 70, 190]), y=y)
    qig.attend_prompt(q, k, v, ints([5, 70, 190]), y=wide[:, :, 4:84])
    assert (y[:5] == 7).all() and (y[190:] == 7).all() and not (y[5:190] == 7).any()
    assert torch.equal(wide[:, :, 4:84], y) and (wide[:, :, :4] == 7).all() and (wide[:, :, 84:] == 7).all()
    w, al = want(q[5:190], k[5:190], v[5:190], [65, 120], [65, 120], True, 1 / math.sqrt(80), dtype, dtype)
    ref.check(y[5:190], w, al)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_unseen_places_hold_anything(dtype, bad):
    """NaN and infinities in later keys and in other sequences' rows."""
    lens = [40, 90]
    q, k, v = make(lens, lens, 2, 1, 64, dtype, 1)
    st = ints([0, 40, 130])
    clean = qig.attend_prompt(q, k, v, st)
    k[100:], v[100:] = bad, bad     # positions from 60 on of the second
    y = qig.attend_prompt(q, k, v, st)
    assert torch.equal(y[:100], clean[:100])
    # the tensors' tails behind the last sequence as well
    y = qig.attend_prompt(q, k, v, ints([0, 40, 100]))
    assert torch.equal(y[:100], clean[:100])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_nan_is_seen(dtype):
    q, k, v = make([70], [70], 2, 1, 64, dtype, 1)
    k[50, 0, 3] = math.nan
    v[60, 0, 5] = math.nan
    y = qig.attend_prompt(q, k, v, ints([0, 70])).isnan()
    assert not y[:50].any() and y[50:].all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_far_scores(dtype):
    """Scores hundreds apart in growing order, so that the maximum moves at every step,
    and of the lowest values that a type has."""
    n, d = 300, 64
    q = torch.zeros((n, 1, d), dtype=dtype, device="cuda")
    k = torch.zeros((n, 1, d), dtype=dtype, device="cuda")
    q[:, 0, 0] = 8
    k[:, 0, 0] = torch.arange(n, device="cuda").to(dtype)
    v = torch.randn((n, 1, d), generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    st = ints([0, n])
    for sign in (1, -1):
        y = qig.attend_prompt(q, k * sign, v, st, scale=1.0)
        w, al = want(q, k * sign, v, [n], [n], True, 1.0, dtype, dtype)
        ref.check(y, w, al)


def test_largest_offsets():
    """Rows behind 2^32 bytes and 2^31 elements from the tensor's start."""
    hq, hkv, d, n = 2, 1, 64, 100
    far = 36 << 20                                   # elements between tokens
    q, k, v = make([n], [n], hq, hkv, d, BF16, 1)
    big = torch.empty((n - 1) * far + hq * d, dtype=BF16, device="cuda")
    put = lambda t, h: big.as_strided((n, h, d), (far, d, 1)).copy_(t)  # noqa: E731
    st = ints([0, n])
    y = qig.attend_prompt(q, k, v, st)
    assert torch.equal(qig.attend_prompt(put(q, hq), k, v, st), y)
    assert torch.equal(qig.attend_prompt(q, put(k, hkv), v, st), y)
    assert torch.equal(qig.attend_prompt(q, k, put(v, hkv), st), y)
    assert torch.equal(qig.attend_prompt(q, k, v, st, y=big.as_strided((n, hq, d), (far, d, 1))), y)


def test_wrong_starts_stay_inside():
    """Starts that decrease or leave the tensors touch nothing outside of them."""
    q, k, v = make([60], [60], 2, 1, 64, BF16, 1)
    y = torch.full((80, 2, 64), 5.0, dtype=BF16, device="cuda")
    for st in ([0, 500], [-40, 30, 20, 70], [50, 10, -3], [2147483647, -2147483648], [0, 2147483647]):
        qig.attend_prompt(q, k, v, ints(st), y=y[10:70])
        torch.cuda.synchronize()
        assert (y[:10] == 5).all() and (y[70:] == 5).all()
