"""The attention operators as a server uses them: with the int8 linear layer's
products, on streams of their own, in graphs, and one after the other."""
import math

import numpy as np
import pytest
import torch

import attend_ref as ref
import quant_integer_gemm_amd as qig

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


class Server:
    """Weights of one layer's q, k and v in int8, and a pool of pages."""

    def __init__(self, rows=6, width=8, npages=40, page=32, hq=4, hkv=2, d=64, hidden=96, dtype=BF16):
        self.hq, self.hkv, self.d, self.page, self.dtype = hq, hkv, d, page, dtype
        self.W, self.sw = qig.quantize_i8(randn(((hq + 2 * hkv) * d, hidden), 1) / math.sqrt(hidden))
        self.pages = qig.new_kv4(npages, hkv, d, page)
        self.pages.fill_(0xff)
        self.tables = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.refs = ints([0] * rows), ints([0] * npages)
        self.ws = qig.new_workspace("cuda")

    def qkv(self, x):
        q, s = qig.quantize_i8(x)
        y = qig.mm_i8(self.W, self.sw, q, s, dtype=self.dtype)
        cut = [self.hq * self.d, self.hkv * self.d, self.hkv * self.d]
        return [p.unflatten(1, (-1, self.d)) for p in y.split(cut, 1)]

    def step(self, x, grown, starts=None):
        """New tokens x of all rows, grown[row] each."""
        self.lengths += grown
        missing = qig.take_pages(self.tables, self.lengths, self.refs, self.page)
        q, k, v = self.qkv(x)
        qig.write_kv4(k, v, self.pages, self.tables, self.lengths, starts)
        return qig.attend_kv4(q, self.pages, self.tables, self.lengths, starts, ws=self.ws), missing


def test_a_request_s_life():
    """Prompts of different lengths, a fork, decoding, a later part of a prompt, compaction,
    and the end: every attention against the formula over the values that were written."""
    s = Server()
    seen = [[] for _ in range(6)]                   # (k, v) as the cache stands for them
    lens = [70, 1, 0, 33, 0, 0]
    starts = ints([0, 70, 71, 71, 104, 104, 104])

    def note(k, v, counts, at=0):
        k, v = (ref.stands_for(t.float().cpu().numpy()) for t in (k, v))
        for r, n in enumerate(counts):
            seen[r].append((k[at:at + n], v[at:at + n]))
            at += n

    def want(row, q, n):
        k, v = (torch.from_numpy(np.concatenate([p[i] for p in seen[row]])) for i in (0, 1))
        total = k.shape[0]
        y, mag, amax = ref.attention(q, k, v, n, [total - n + i for i in range(n)], 1 / 8)
        # |m| + s c is at most 3 |x| largest of the group: the sizes' bounds by the row's largest values
        kq, vq = ref.quantize4(k.numpy()), ref.quantize4(v.numpy())
        ka = torch.from_numpy(ref.values4(kq[0], kq[1], np.abs(kq[2]))).double().repeat_interleave(s.hq // s.hkv, 1)
        va = torch.from_numpy(ref.values4(vq[0], vq[1], np.abs(vq[2])))
        _, mag, _ = ref.attention(q, k, va, n, [total - n + i for i in range(n)], 1 / 8)
        amax = torch.einsum("ihd,jhd->ihj", q.double().abs().cpu(), ka).amax(2, keepdim=True) / 8
        amp = float(q.double().abs().max()) * float(ka.sum(2).max()) / 8
        return y, ref.kv4_allowance(q, mag, amax, amp, s.d, total, s.dtype, s.dtype, float(vq[1].max()))(y)

    # the prompts: exact keys and values for their own attention, the 4-bit ones for later
    x = randn((104, 96), 2, BF16)
    s.lengths += ints(lens)
    assert int(qig.take_pages(s.tables, s.lengths, s.refs, s.page)) == 0
    q, k, v = s.qkv(x)
    y = qig.attend_prompt(q, k, v, starts)
    at = 0
    for n in lens:
        w, mag, amax = ref.attention(q[at:at + n], k[at:at + n], v[at:at + n], n, list(range(n)), 1 / 8)
        ref.check(y[at:at + n], w, ref.allowance(w, mag, amax, s.d, n, 2.0 ** -8, BF16), f"prompt of {n}")
        at += n
    qig.write_kv4(k, v, s.pages, s.tables, s.lengths, starts)
    note(k, v, lens)
    # two rows fork from the first; then all live rows get a token, and the fourth three more
    assert int(qig.fork_pages(s.pages, s.tables, s.lengths, s.refs, ints([0, 0]), ints([2, 4]), s.page)) == 0
    seen[2], seen[4] = list(seen[0]), list(seen[0])
    assert s.refs[s.tables[0, 0]] == 3 and s.refs[s.tables[0, 2]] == 1
    for turn in range(40):
        counts = [1, 1, 1, 4 if turn == 3 else 1, 1, 0]
        at = [sum(counts[:i]) for i in range(7)]
        x = randn((at[-1], 96), 10 + turn, BF16)
        q, k, v = s.qkv(x)
        y, missing = s.step(x, ints(counts), ints(at))
        assert int(missing) == 0
        note(k, v, counts)
        if turn % 13 == 3:
            for r, n in enumerate(counts):
                if n:
                    w, allow = want(r, q[at[r]:at[r + 1]], n)
                    ref.check(y[at[r]:at[r + 1]], w, allow, f"turn {turn}, row {r}")
        if turn == 20:
            qig.free_pages(s.tables, s.lengths, s.refs, ints([1]))
            seen[1] = []
            qig.compact_pages(s.pages, s.tables, s.refs)
    used = int(qig.compact_pages(s.pages, s.tables, s.refs))
    assert used == int((s.refs > 0).sum()) == int((s.refs[:used] > 0).sum())
    # the next part of the fourth's prompt: its prefix read back, exact keys for itself
    n, total = 20, int(s.lengths[3])
    kc, vc = qig.read_kv4(s.pages, s.tables[3:4], s.lengths[3:4], s.d, ints([0, total]), total, dtype=BF16)
    assert torch.equal(kc.cpu(), torch.from_numpy(np.concatenate([p[0] for p in seen[3]])).to(BF16))
    q, k, v = s.qkv(randn((n, 96), 99, BF16))
    kk, vv = torch.cat([kc, k]), torch.cat([vc, v])
    y = qig.attend_prompt(q, kk, vv, ints([0, n]), ints([0, total + n]))
    w, mag, amax = ref.attention(q, kk, vv, n, [total + i for i in range(n)], 1 / 8)
    ref.check(y, w, ref.allowance(w, mag, amax, s.d, total + n, 2.0 ** -8, BF16))
    qig.free_pages(s.tables, s.lengths, s.refs, ints([0, 1, 2, 3, 4, 5]))
    assert not s.refs.any() and (s.tables == -1).all() and not s.lengths.any()


def test_captured_decoding():
    """A decoding step in a graph, on inputs that change, with eager steps of another
    server and synchronizations between the replays."""
    a, b = Server(), Server()
    prompt, starts = randn((100, 96), 1, BF16), ints([0, 50, 60, 60, 100, 100, 100])
    for s in (a, b):
        s.step(prompt, ints([50, 10, 0, 40, 0, 0]), starts)
    one = ints([1, 1, 1, 1, 0, 1])
    at = ints([0, 1, 2, 3, 4, 4, 5])
    x = randn((5, 96), 2, BF16)
    held = [t.clone() for t in (a.tables, a.lengths, a.refs, a.pages)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.step(x, one, at)
    torch.cuda.current_stream().wait_stream(side)
    for t, h in zip((a.tables, a.lengths, a.refs, a.pages), held):
        t.copy_(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, missing = a.step(x, one, at)
    for t, h in zip((a.tables, a.lengths, a.refs, a.pages), held):
        t.copy_(h)
    for i in range(40):
        x.copy_(randn((5, 96), 50 + i, BF16))
        graph.replay()
        want, gone = b.step(x, one, at)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and int(missing) == int(gone)
        for t, u in zip((a.tables, a.lengths, a.refs, a.pages), (b.tables, b.lengths, b.refs, b.pages)):
            assert torch.equal(t, u)


def test_captured_prompts():
    """One graph, replayed on packed prompts of other lengths."""
    q, k, v = randn((300, 4, 64), 1, F16), randn((300, 2, 64), 2, F16), randn((300, 2, 64), 3, F16)
    starts = ints([0, 100, 300])
    qig.attend_prompt(q, k, v, starts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = qig.attend_prompt(q, k, v, starts)
    for s in ([0, 100, 300], [0, 0, 300], [0, 299, 300], [0, 1, 2]):
        starts.copy_(ints(s))
        graph.replay()
        want = qig.attend_prompt(q, k, v, starts)
        torch.cuda.synchronize()
        assert torch.equal(y[:s[-1]], want[:s[-1]])


def test_two_graphs_with_default_workspaces():
    """Each capture has its own; replayed at the same time on two streams."""
    torch.manual_seed(1)
    n, d = 9000, 128
    pages = qig.new_kv4(2 * 141, 2, d, 64)
    tables = ints([list(range(141)), list(range(141, 282))])
    lengths = ints([n, n])
    kv = torch.randn((2 * n, 2, d), device="cuda")
    qig.write_kv4(kv, kv, pages, tables, lengths, ints([0, n, 2 * n]))
    qs = [torch.randn((2, 14, d), device="cuda").bfloat16() for _ in range(2)]
    want = [qig.attend_kv4(q, pages, tables, lengths, ws=qig.workspace(q.device)) for q in qs]
    streams, graphs, ys = [torch.cuda.Stream() for _ in range(2)], [], []
    torch.cuda.synchronize()
    for q, st in zip(qs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            ys.append(qig.attend_kv4(q, pages, tables, lengths, ws=qig.workspace(q.device)))
        graphs.append(graph)
    for _ in range(10):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, want))


def test_given_streams():
    """Every call on a stream of its own, given as an object or by its handle alone."""
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    s = Server()
    x = randn((90, 96), 1, BF16)
    starts = ints([0, 40, 90])
    q, k, v = (t.contiguous() for t in s.qkv(x))
    lengths, refs = ints([40, 50, 0]), ints([0] * 40)

    def all_calls(st):
        tables = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
        pages = qig.new_kv4(40, 2, 64, 32)
        pages.zero_()
        lens, rf, to = lengths.clone(), refs.clone(), torch.empty(40, dtype=torch.int32, device="cuda")
        parents, children, rows = ints([0]), ints([2]), ints([1])
        src, dst, two = ints([0]), ints([30]), ints([0, 40, 90, 90])
        torch.cuda.synchronize()
        kw = {} if st is None else {"stream": st}
        out = [qig.take_pages(tables, lens, rf, 32, **kw), qig.attend_prompt(q, k, v, starts, **kw)]
        qig.write_kv4(k, v, pages, tables, lens, two, **kw)
        out += list(qig.read_kv4(pages, tables, lens, 64, two, 90, **kw))
        out.append(qig.fork_pages(pages, tables, lens, rf, parents, children, 32, **kw))
        out.append(qig.attend_kv4(q[:3], pages, tables, lens, ws=s.ws, **kw))
        qig.copy_pages(pages, src, dst, **kw)
        qig.free_pages(tables, lens, rf, rows, **kw)
        out += [qig.compact_pages(pages, tables, rf, to=to, **kw), tables, lens, rf, to, pages]
        torch.cuda.synchronize()
        return out

    want = all_calls(None)
    other = torch.cuda.Stream()
    for st in (other, Handle(other)):
        for a, b in zip(all_calls(st), want):
            assert torch.equal(a, b)
