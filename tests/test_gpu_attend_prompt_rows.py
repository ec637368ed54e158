"""attend_prompt where few rows meet many keys, which splits the keys, and where many
sequences fill the GPU, which does not: both against the 64-bit form."""
import math

import pytest
import torch

import attend_ref as ref
import quant_integer_gemm_amd as qig
from test_gpu_attend_prompt import BF16, F16, F32, ints, make, run, starts_of, want

pytestmark = pytest.mark.gpu

TYPES = [F32, BF16, F16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nk", [65, 96, 127, 128, 129, 191, 256, 257, 383, 511, 512, 513, 2000])
def test_one_query_on_many_keys(nk, dtype):
    run([1], [nk], 4, 2, 128, dtype, True, nk)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [8, 64, 72, 128, 200, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_few_queries_on_many_keys(d, dtype, causal):
    run([9, 0, 33], [700, 5, 300], 6, 2, d, dtype, causal, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 72, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences_fill_the_card(d, dtype, causal):
    """Tiles of 128 rows: 64 short sequences of 8 key heads."""
    lens = [(i * 5) % 11 for i in range(64)]
    klens = [n + (i * 37) % 200 for i, n in enumerate(lens)]
    run(lens, klens, 16, 8, d, dtype, causal, d)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_sequences_fill_the_card(dtype):
    """Several tiles and many steps a sequence: 7 x 300 queries of 24 heads."""
    run([300] * 7, [300, 310, 420, 300, 555, 300, 301], 24, 24, 64, dtype, True, 7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("many", [False, True])
def test_unseen_places(dtype, bad, many):
    """NaN and infinities in keys and values that only the last queries see."""
    lens = [40, 200] + ([3] * 60 if many else [])
    hq, hkv = (16, 8) if many else (2, 1)
    q, k, v = make(lens, lens, hq, hkv, 64, dtype, 1)
    st = ints(starts_of(lens))
    clean = qig.attend_prompt(q, k, v, st)
    k[190:240], v[190:240] = bad, bad            # positions from 150 on of the second
    y = qig.attend_prompt(q, k, v, st)
    assert torch.equal(y[:190], clean[:190]) and torch.equal(y[240:], clean[240:])
    assert y[190:240].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("many", [False, True])
def test_a_nan_reaches_who_sees_it(dtype, many):
    lens = [300] + ([3] * 60 if many else [])
    hq, hkv = (16, 8) if many else (2, 1)
    q, k, v = make(lens, lens, hq, hkv, 64, dtype, 1)
    k[150, 0, 3] = math.nan
    v[20, 0, 5] = math.nan
    y = qig.attend_prompt(q, k, v, ints(starts_of(lens))).isnan()
    assert not y[:20].any() and y[150:300, 0].all() and not y[300:].any()
    assert y[20:150, 0, 5].all() and not y[20:150, 0, 6:].any()
    assert not y[:300, hq // hkv:].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("many", [False, True])
def test_scores_that_grow_and_fall(dtype, many):
    """The maximum stands with another step, and so another wave, for every sign."""
    lens = [5] * (64 if many else 1)
    klens = [900] + [6] * (len(lens) - 1)
    hkv = 8 if many else 1
    q, k, v = make(lens, klens, hkv, hkv, 64, dtype, 3)
    q[:] = 0
    k[:] = 0
    q[:, :, 0] = 8
    k[:900, :, 0] = (torch.arange(900, device="cuda") / 4).to(dtype)[:, None]
    st, kst = ints(starts_of(lens)), ints(starts_of(klens))
    for sign in (1, -1):
        y = qig.attend_prompt(q, k * sign, v, st, kst, scale=1.0)
        w, al = want(q, k * sign, v, lens, klens, True, 1.0, dtype, dtype)
        ref.check(y, w, al)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 72])
def test_few_queries_in_a_graph(dtype, d):
    q, k, v = make([20], [600], 4, 2, d, dtype, 1)
    st, kst = ints([0, 20]), ints([0, 600])
    y = torch.empty_like(q)
    qig.attend_prompt(q, k, v, st, kst, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qig.attend_prompt(q, k, v, st, kst, y=y)
    for n in (600, 333, 20, 0):
        kst.copy_(torch.tensor([0, n], dtype=torch.int32))
        want_ = qig.attend_prompt(q, k, v, st, kst)
        y.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [8, 40, 64, 72, 96, 128, 136])
@pytest.mark.parametrize("many", [False, True])
def test_a_key_at_minus_infinity(dtype, d, many):
    """A channel of a key at -infinity, positive in all queries: the key counts for nothing."""
    lens = [150] + ([3] * 60 if many else [])
    hq, hkv = (16, 8) if many else (2, 1)
    q, k, v = make(lens, lens, hq, hkv, d, dtype, d)
    q[:, :, 0] = q[:, :, 0].abs() + 1
    k[70:73, 0, 0] = -math.inf
    y = qig.attend_prompt(q, k, v, ints(starts_of(lens)))
    k[70:73, 0] = 0
    k[70:73, 0, 0] = -60000                     # far below all others: 0 in 64 bits too
    w, al = want(q, k, v, lens, lens, True, 1 / math.sqrt(d), dtype, dtype)
    ref.check(y, w, al)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [40, 80, 96, 128, 136])
@pytest.mark.parametrize("many", [False, True])
def test_odd_addresses(dtype, d, many):
    """Rows that no 16-byte copy can take give the results of those that one can."""
    lens = [200, 70] + ([3] * 60 if many else [])
    hq, hkv = (16, 8) if many else (2, 1)
    q, k, v = make(lens, lens, hq, hkv, d, dtype, d)
    wide = torch.full((sum(lens), hkv * d * 2 + 3), math.nan, dtype=dtype, device="cuda")
    ko, vo = (wide[:, i:i + hkv * d].unflatten(1, (hkv, d)) for i in (1, hkv * d + 3))
    ko.copy_(k)
    vo.copy_(v)
    y = qig.attend_prompt(q, ko, vo, ints(starts_of(lens)))
    w, al = want(q, k, v, lens, lens, True, 1 / math.sqrt(d), dtype, dtype)
    ref.check(y, w, al)
