"""The attention operators without a GPU: argument checks of the C ABI and of the
binding, and the plain forms of the tests against hand-made cases."""
import ctypes

import numpy as np
import pytest

import attend_ref as ref
import quant_integer_gemm_amd as qig

torch = pytest.importorskip("torch")

P = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)   # 8-byte aligned only
FOUR = ctypes.c_void_p(0x10004)
ODD = ctypes.c_void_p(0x10001)
BIG = 1 << 31


def _prompt(**kw):
    a = dict(q=P, qn=256, qh=64, k=P, kn=128, kh=64, v=P, vn=128, vh=64, t=0, nt=5, nk=5, hq=4, hkv=2, d=64, st=P, kst=P,
             nseq=1, causal=1, scale=0.0, y=P, yn=256, yh=64, yt=0)
    a.update(kw)
    return qig.load().attend_prompt(*a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(t=3), -1), (dict(t=-1), -1), (dict(yt=3), -1), (dict(nt=-1), -1), (dict(nt=BIG), -1), (dict(nk=-1), -1),
    (dict(nk=BIG), -1), (dict(hq=5), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(hq=2048, hkv=1024), -1),
    (dict(d=0), -1), (dict(d=60), -1), (dict(d=264), -1), (dict(nseq=-1), -1), (dict(nseq=BIG - 1), -1),
    (dict(causal=2), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(qn=-1), -1), (dict(kh=-64), -1), (dict(vn=-1), -1), (dict(yh=-1), -1), (dict(q=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(st=None), -1), (dict(kst=None), -1), (dict(y=None), -1), (dict(q=FOUR), None),
    (dict(q=ODD), -2), (dict(k=ODD, t=1), -2), (dict(v=ODD), -2), (dict(y=ODD, yt=2), -2), (dict(st=ODD), -2),
    (dict(kst=ODD), -2), (dict(nt=0), 0), (dict(nseq=0), 0), (dict(nt=0, q=None, y=None), 0),
    (dict(nt=1 << 30, hq=1024, hkv=1), -1),          # more tiles than a launch holds
])
def test_attend_prompt_argument_checks(kw, rc):
    if rc is not None:
        assert _prompt(**kw) == rc


CACHE = dict(hkv=2, d=64, pages=P, npages=9, ps=5120, page=32, tables=P, ld=4, width=4, lengths=P, starts=P, nseq=3)
BAD_CACHE = [
    (dict(d=96), -1), (dict(d=32), -1), (dict(hkv=0), -1), (dict(hkv=1025), -1), (dict(npages=-1), -1),
    (dict(npages=BIG), -1), (dict(ps=5104), -1), (dict(ps=5128), -2), (dict(page=16), -1), (dict(page=48), -1),
    (dict(page=0), -1), (dict(page=1 << 17), -1), (dict(ld=3), -1), (dict(width=-1), -1), (dict(width=BIG, ld=BIG), -1),
    (dict(nseq=-1), -1), (dict(pages=None), -1), (dict(pages=MIS), -2), (dict(tables=None), -1), (dict(tables=ODD), -2),
    (dict(lengths=None), -1), (dict(lengths=ODD), -2), (dict(starts=ODD), -2), (dict(starts=None), -1),
    (dict(nt=-1), -1), (dict(nt=BIG), -1), (dict(t=4), -1), (dict(nt=0), 0), (dict(nseq=0), 0),
]


def _split(kw, first):
    a, c = dict(first), dict(CACHE)
    for name, v in kw.items():
        (a if name in a else c)[name] = v
    return a, c


@pytest.mark.parametrize("fn", ["write_kv4", "read_kv4"])
@pytest.mark.parametrize("kw,rc", BAD_CACHE + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=ODD), -2), (dict(v=ODD, t=1), -2), (dict(kn=-1), -1), (dict(vh=-1), -1)])
def test_rows_argument_checks(fn, kw, rc):
    a, c = _split(kw, dict(k=P, kn=128, kh=64, v=P, vn=128, vh=64, t=0, nt=5))
    assert getattr(qig.load(), fn)(*a.values(), *c.values(), None) == rc


@pytest.mark.parametrize("kw,rc", BAD_CACHE + [
    (dict(q=None), -1), (dict(q=ODD), -2), (dict(y=None), -1), (dict(y=ODD), -2), (dict(yt=9), -1), (dict(hq=3), -1),
    (dict(scale=-0.5), -1), (dict(scale=float("nan")), -1), (dict(ws=MIS), -2), (dict(qn=-1), -1), (dict(yn=-1), -1)])
def test_attend_kv4_argument_checks(kw, rc):
    end = dict(scale=0.0, y=P, yn=256, yh=64, yt=0, ws=None)
    late = {n: kw[n] for n in kw if n in end}
    a, c = _split({n: v for n, v in kw.items() if n not in end}, dict(q=P, qn=256, qh=64, t=0, nt=5, hq=4))
    end.update(late)
    assert qig.load().attend_kv4(*a.values(), *c.values(), *end.values(), None) == rc


def test_sizes():
    lib = qig.load()
    assert lib.kv4_page_bytes(32, 1, 64) == 32 * 80 and qig.kv4_page_bytes(64, 4, 128) == 64 * 4 * 160
    for bad in ((0, 1, 64), (33, 1, 64), (32, 0, 64), (32, 1, 80), (1 << 17, 1, 64)):
        assert lib.kv4_page_bytes(*bad) == 0
    assert lib.pages_scratch_bytes(1, 0) >= 8 and lib.pages_scratch_bytes(65, 3) >= 28
    for bad in ((0, 1), (-1, 1), ((1 << 20) + 1, 1), (5, -1), (5, BIG)):
        assert lib.pages_scratch_bytes(*bad) == 0


POOL = dict(tables=P, rows=4, ld=8, width=8, lengths=P, refs=P, npages=20)
BAD_POOL = [
    (dict(rows=-1), -1), (dict(width=-1), -1), (dict(ld=7), -1), (dict(npages=0), -1), (dict(npages=(1 << 20) + 1), -1),
    (dict(rows=1 << 20, width=1 << 11, ld=1 << 11), -1), (dict(rows=BIG), -1), (dict(tables=None), -1),
    (dict(tables=ODD), -2), (dict(refs=None), -1), (dict(refs=ODD), -2),
]


@pytest.mark.parametrize("kw,rc", BAD_POOL + [
    (dict(which=None), -1), (dict(which=ODD), -2), (dict(n=-1), -1), (dict(n=BIG), -1), (dict(lengths=None), -1),
    (dict(n=0), 0), (dict(rows=0), 0)])
def test_free_pages_argument_checks(kw, rc):
    a = {**POOL, "which": P, "n": 2, **kw}
    assert qig.load().free_pages(*a.values(), None) == rc


@pytest.mark.parametrize("kw,rc", BAD_POOL + [
    (dict(page=0), -1), (dict(page=BIG), -1), (dict(missing=None), -1), (dict(missing=ODD), -2), (dict(scratch=None), -1),
    (dict(scratch=FOUR), -2), (dict(lengths=None), -1), (dict(lengths=ODD), -2)])
def test_take_pages_argument_checks(kw, rc):
    a = {**POOL, "page": 32, "missing": P, "scratch": P, **kw}
    assert qig.load().take_pages(*a.values(), None) == rc


BAD_PAGES = [(dict(pages=None), -1), (dict(pages=MIS), -2), (dict(nbytes=0), -1), (dict(nbytes=24), -2),
             (dict(step=16), -1), (dict(step=72), -2)]


@pytest.mark.parametrize("kw,rc", BAD_POOL + BAD_PAGES + [
    (dict(page=0), -1), (dict(parents=None), -1), (dict(children=None), -1), (dict(parents=ODD), -2),
    (dict(children=ODD), -2), (dict(n=-1), -1), (dict(n=BIG), -1), (dict(missing=None), -1), (dict(scratch=FOUR), -2),
    (dict(lengths=None), -1)])
def test_fork_pages_argument_checks(kw, rc):
    a = {"pages": P, "nbytes": 64, "step": 64, **POOL, "page": 32, "parents": P, "children": P, "n": 2, "missing": P,
         "scratch": P, **kw}
    assert qig.load().fork_pages(*a.values(), None) == rc


@pytest.mark.parametrize("kw,rc", BAD_POOL + BAD_PAGES + [
    (dict(used=None), -1), (dict(used=ODD), -2), (dict(to=ODD), -2), (dict(scratch=None), -1), (dict(scratch=FOUR), -2)])
def test_compact_pages_argument_checks(kw, rc):
    a = {"pages": P, "nbytes": 64, "step": 64, **{n: v for n, v in POOL.items() if n != "lengths"}, "used": P, "to": None,
         "scratch": P, **kw}
    assert qig.load().compact_pages(*a.values(), None) == rc


@pytest.mark.parametrize("kw,rc", BAD_PAGES + [
    (dict(npages=-1), -1), (dict(npages=BIG), -1), (dict(src=None), -1), (dict(dst=None), -1), (dict(src=ODD), -2),
    (dict(n=-1), -1), (dict(n=BIG), -1), (dict(n=0), 0), (dict(npages=0, pages=None), 0)])
def test_copy_pages_argument_checks(kw, rc):
    a = {"pages": P, "npages": 20, "nbytes": 64, "step": 64, "src": P, "dst": P, "n": 2, **kw}
    assert qig.load().copy_pages(*a.values(), None) == rc


# --- the binding ------------------------------------------------------------------------------------------------------

def z(*shape, t=torch.float32):
    return torch.zeros(shape, dtype=t)


I32 = torch.int32


def refused(text, fn, *a, **kw):
    with pytest.raises(qig.QigError, match=text):
        fn(*a, **kw)


def test_attend_prompt_binding():
    q, k, st = z(5, 4, 64), z(5, 2, 64), z(2, t=I32)
    f = qig.attend_prompt
    refused("must be a GPU tensor", f, q, k, k, st)
    refused("q must be float32", f, q.double(), k, k, st)
    refused("k must be torch.float32", f, q, k.half(), k, st)
    refused("v must be torch.float32", f, q, k, k.half(), st)
    refused("must be .tokens", f, q[0], k, k, st)
    refused("unit stride", f, q.transpose(1, 2), k, k, st)
    refused("heads of 32", f, q, z(5, 2, 32), k, st)
    refused("v has 1 heads", f, q, k, z(5, 1, 64), st)
    refused("v has 4 tokens", f, q, k, k[:4], st)
    refused("starts must be", f, q, k, k, z(2, t=torch.int64))
    refused("starts must be", f, q, k, k, z(1, 2, t=I32))
    refused("k_starts must be contiguous with 2", f, q, k, k, st, z(3, t=I32))
    refused("scale must be above 0", f, q, k, k, st, scale=0.0)
    refused("scale must be above 0", f, q, k, k, st, scale=float("nan"))
    refused("y holds 4 tokens", f, q, k, k, st, y=z(4, 4, 64))
    refused("y is torch.float16", f, q, k, k, st, y=z(5, 4, 64, t=torch.float16), dtype=torch.float32)
    refused("rows overlap", f, q, k, k, st, y=z(5, 1, 64).expand(5, 4, 64))
    refused("rows overlap", f, q, k, k, st, y=z(1, 4, 64).expand(5, 4, 64))
    refused("rows overlap", f, q, k, k, st, y=z(2000).as_strided((5, 4, 64), (200, 64, 1)))


def test_cache_binding():
    pages, t, n = qig.new_kv4(9, 2, 64, 32, device="cpu"), z(3, 4, t=I32), z(3, t=I32)
    k, q = z(3, 2, 64), z(3, 4, 64)
    assert pages.shape == (9, 2, 2560)
    for bad in ((9, 2, 96), (9, 2, 64, 48), (9, 0, 64), (-1, 2, 64)):
        refused("no cache of", qig.new_kv4, *bad, device="cpu")
    for f, x in ((qig.write_kv4, (k, k)), (qig.attend_kv4, (q,)), (qig.read_kv4, ())):
        d = () if x else (64,)
        refused("must be a GPU tensor", f, *x, pages, t, n, *d)
        refused("pages must be torch.uint8", f, *x, pages.to(I32), t, n, *d)
        refused("pages must be .pages", f, *x, pages[0], t, n, *d)
        refused("pages must be .pages", f, *x, pages[:, :, ::2], t, n, *d)
        refused("no whole blocks", f, *x, pages[:, :, :2480].contiguous(), t, n, *d)
        refused("tables must be torch.int32", f, *x, pages, t.long(), n, *d)
        refused("tables must be 2-D", f, *x, pages, t[0], n, *d)
        refused("tables must be 2-D", f, *x, pages, t.t(), n, *d)
        refused("lengths must be contiguous with 3", f, *x, pages, t, n[:2], *d)
        refused("starts must be contiguous with 4", f, *x, pages, t, n, *d, z(3, t=I32), **({} if x else {"nt": 3}))
    refused("nt is needed", qig.read_kv4, pages, t, n, 64, z(4, t=I32))
    refused("starts says", qig.read_kv4, pages, t, n, 64, nt=5)
    refused("starts says", qig.write_kv4, z(4, 2, 64), z(4, 2, 64), pages, t, n)
    refused("k has 4 heads, pages have 2", qig.write_kv4, q, q, pages, t, n)
    refused("v has 2 tokens", qig.write_kv4, k, k[:2], pages, t, n)
    refused("k holds 2 tokens", qig.read_kv4, pages, t, n, 64, nt=3, k=k[:2])
    refused("ws holds 100 bytes", qig.attend_kv4, q, pages, t, n, ws=z(100, t=torch.uint8))
    refused("scale must be above 0", qig.attend_kv4, q, pages, t, n, scale=-1.0)


def test_pages_binding():
    pages, t, n, refs = z(9, 4, 4), z(3, 4, t=I32), z(3, t=I32), z(9, t=I32)
    one = z(1, t=I32)
    refused("must be a GPU tensor", qig.copy_pages, pages, one, one)
    refused("dst must be contiguous with 1", qig.copy_pages, pages, one, z(2, t=I32))
    refused("src must be torch.int32", qig.copy_pages, pages, one.long(), one)
    refused("each page must be contiguous", qig.copy_pages, pages.transpose(1, 2), one, one)
    refused("pages must have", qig.copy_pages, z(9), one, one)
    refused("must be a GPU tensor", qig.take_pages, t, n, refs, 32)
    refused("must be a GPU tensor", qig.free_pages, t, n, refs, one)
    refused("must be a GPU tensor", qig.fork_pages, pages, t, n, refs, one, one, 32)
    refused("must be a GPU tensor", qig.compact_pages, pages, t, refs)
    refused("rows must be", qig.free_pages, t, n, refs, z(1, 1, t=I32))
    refused("lengths must be", qig.free_pages, t, n[:1], refs, one)
    refused("refs must be torch.int32", qig.take_pages, t, n, refs.long(), 32)
    refused("refs must be a contiguous", qig.take_pages, t, n, z(9, 2, t=I32)[:, 0], 32)
    refused("missing must be", qig.take_pages, t, n, refs, 32, missing=z(2, t=I32))
    refused("no pool of 0 pages", qig.take_pages, t, n, refs[:0], 32)
    refused("refs counts 8 pages", qig.fork_pages, pages, t, n, refs[:8], one, one, 32)
    refused("refs counts 8 pages", qig.compact_pages, pages, t, refs[:8])
    refused("children must be", qig.fork_pages, pages, t, n, refs, one, z(2, t=I32), 32)
    refused("to must be", qig.compact_pages, pages, t, refs, to=z(8, t=I32))


# --- the tests' plain forms -----------------------------------------------------------------------------------------

def test_quantize4_by_hand():
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :16] = np.arange(16)
    x[0, 16] = 2.5                                   # halfway: up
    c, s, m = ref.quantize4(x)
    assert s[0, 0] == 1 and m[0, 0] == 0 and list(c[0, 0, :17]) == list(range(16)) + [3] and not c[0, 0, 17:].any()
    x[0] = -1.00390625                               # between two bf16
    c, s, m = ref.quantize4(x)
    assert m[0, 0] == -1.0078125 and s[0, 0] * 15 >= 0.00390625 and np.abs(ref.values4(c, s, m) - x).max() <= s[0, 0] / 2
    x[0] = 7.0
    c, s, m = ref.quantize4(x)
    assert s[0, 0] == 0 and (ref.stands_for(x) == 7).all()


def test_bf16_steps():
    r = np.random.RandomState(1)
    x = np.concatenate([r.randn(5000), r.randn(500) * 1e-39, [0.0, 1.0, -1.0, 3.0]]).astype(np.float32)
    down, up = ref.bf16_floor(x), ref.bf16_ceil(np.abs(x).astype(np.float64))
    for y in (down, up):
        assert not (y.view(np.uint32) & 0xffff).any()
    nxt = lambda y, to: torch.nextafter(torch.from_numpy(y).to(torch.bfloat16), torch.tensor(to, dtype=torch.bfloat16)).float().numpy()  # noqa: E731,E501
    assert (down <= x).all() and (nxt(down, np.inf) > x).all()
    assert (up >= np.abs(x)).all() and ((nxt(up, -np.inf) < np.abs(x)) | (up == 0)).all()


def test_attention_by_hand():
    q = torch.ones((1, 1, 8))
    k = torch.zeros((3, 1, 8))
    k[1] = np.log(3.0) / 8
    v = torch.arange(24.0).view(3, 1, 8)
    y, mag, _ = ref.attention(q, k, v, 1, [2], 1.0)
    assert torch.allclose(y[0, 0], (v[0, 0] + 3 * v[1, 0] + v[2, 0]).double() / 5, atol=1e-6)
    y, _, _ = ref.attention(q, k, v, 1, [-1], 1.0)
    assert (y == 0).all()
    y, _, _ = ref.attention(q, k, v, 1, [2], 1.0, torch.tensor([True, False, False]))
    assert torch.equal(y[0, 0], v[0, 0].double())


def test_pool_by_hand():
    p = ref.Pool([[2, 0], [-1, -1], [-1, -1]], [5, 0, 0], [1, 0, 1, 0, 0])
    assert p.fork([0], [1], 4) == (0, [(0, 1)])
    assert p.t[1] == [2, 1] and p.refs == [1, 1, 2, 0, 0] and p.len[1] == 5
    p.free([0, 0])
    assert p.refs == [0, 1, 1, 0, 0]
    p.len[2] = 8
    assert p.take(4) == 0 and p.t[2] == [0, 3]
    p.free([1])
    assert p.compact() == (2, [0, 1, 2, 1, 4], [(3, 1)]) and p.t[2] == [0, 1]


# The packed calls with their words; nt = 0 (or no pairs), so that valid ones return before a launch.
PACKED = {
    0: [P, 256, 64, P, 128, 64, P, 128, 64, 0, 0, 5, 4, 2, 64, P, P, 1, 1, 0.0, P, 256, 64, 0],
    1: [P, 128, 64, P, 128, 64, 0, 0, 2, 64, P, 9, 5120, 32, P, 4, 4, P, P, 3],
    2: [P, 128, 64, P, 128, 64, 0, 0, 2, 64, P, 9, 5120, 32, P, 4, 4, P, P, 3],
    3: [P, 256, 64, 0, 0, 4, 2, 64, P, 9, 5120, 32, P, 4, 4, P, P, 3, 0.0, P, 256, 64, 0, None],
    4: [P, 20, 64, 64, P, P, 0],
    5: [P, 4, 8, 8, P, P, 20, P, 0],
}


def _packed(op, words, **at):
    import struct
    words = list(words)
    for i, v in at.items():
        words[int(i[1:])] = v
    raw = b"".join(struct.pack("=d" if isinstance(w, float) else "=q",
                               w.value if isinstance(w, ctypes.c_void_p) else 0 if w is None else w) for w in words)
    return qig.load().qig_attend_packed(op, raw, None)


@pytest.mark.parametrize("op", sorted(PACKED))
def test_packed_calls_take_their_words(op):
    assert _packed(op, PACKED[op]) == 0
    bad = {0: dict(_10=-1), 1: dict(_7=-1), 2: dict(_8=0), 3: dict(_7=96), 4: dict(_6=-1), 5: dict(_8=-1)}[op]
    assert _packed(op, PACKED[op], **bad) == -1


def test_packed_calls_refuse_what_does_not_fit():
    w = PACKED[0]
    assert _packed(-1, w) == -1 and _packed(9, w) == -1 and qig.load().qig_attend_packed(0, None, None) == -1
    for i in ("_9", "_18", "_23"):                       # a type, causal, the result's type
        assert _packed(0, w, **{i: 1 << 32}) == -1 and _packed(0, w, **{i: -(1 << 40)}) == -1
    assert _packed(0, w, _19=1e-30) == 0
    for scale in (1e-50, 1e31, 1e300, -1e-50, float("nan"), float("inf")):
        assert _packed(0, w, _19=scale) == -1            # 1e-50 is 0 in fp32, which would ask for 1 / sqrt(d)
        assert _packed(3, PACKED[3], _18=scale) == -1
