"""The pages' operators against lists: every result is whole numbers and has to be equal."""
import random

import pytest
import torch

import attend_ref as ref
import quant_integer_gemm_amd as qig

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def new_pages(npages, words, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-(1 << 31), (1 << 31) - 1, (npages, words), generator=g, dtype=torch.int32).cuda()


class Both:
    """A pool on the GPU and as lists."""

    def __init__(self, rows, width, npages, page, seed, words=8, fill=0.6, ld=None):
        rng = random.Random(seed)
        order = list(range(npages))
        rng.shuffle(order)
        t, lens, refs = [[-1] * width for _ in range(rows)], [0] * rows, [0] * npages
        for r in range(rows):
            n = rng.randint(0, width)
            if rng.random() > fill or len(order) < n:
                continue
            lens[r] = max(0, n * page - rng.randrange(page))
            for c in range(-(-lens[r] // page)):
                t[r][c] = order.pop()
                refs[t[r][c]] = 1
        self.page, self.rng, self.width = page, rng, width
        self.ref = ref.Pool(t, lens, refs)
        store = torch.full((rows, ld or width), 77, dtype=torch.int32, device="cuda")
        self.t = store[:, :width]
        if rows and width:
            self.t.copy_(ints(t))
        self.store, self.len, self.refs = store, ints(lens), ints(refs)
        self.pages = new_pages(npages, words, seed)
        self.held = self.pages.clone()

    def same(self):
        torch.cuda.synchronize()
        assert self.t.tolist() == self.ref.t
        assert self.len.tolist() == self.ref.len
        assert self.refs.tolist() == self.ref.refs
        assert torch.equal(self.pages, self.held)
        assert (self.store[:, self.width:] == 77).all()

    def copied(self, pairs):
        if pairs:
            a, b = zip(*pairs)
            self.held[list(b)] = self.held[list(a)]

    def free(self, rows):
        qig.free_pages(self.t, self.len, self.refs, ints(rows))
        self.ref.free(rows)
        self.same()

    def take(self):
        got = qig.take_pages(self.t, self.len, self.refs, self.page)
        assert int(got) == self.ref.take(self.page)
        self.same()

    def fork(self, parents, children):
        got = qig.fork_pages(self.pages, self.t, self.len, self.refs, ints(parents), ints(children), self.page)
        missing, pairs = self.ref.fork(parents, children, self.page)
        self.copied(pairs)
        assert int(got) == missing
        self.same()

    def compact(self):
        to = torch.empty(len(self.ref.refs), dtype=torch.int32, device="cuda")
        got = qig.compact_pages(self.pages, self.t, self.refs, to=to)
        used, want, pairs = self.ref.compact()
        self.copied(pairs)
        assert int(got) == used and to.tolist() == want
        self.same()

    def grow(self, most):
        grown = [max(0, min(n + self.rng.randint(0, most), self.width * self.page + 3)) for n in self.ref.len]
        self.ref.len = grown
        self.len.copy_(ints(grown))


SIZES = [(1, 1, 1, 1), (4, 3, 20, 32), (9, 70, 300, 16), (40, 17, 64, 5), (33, 200, 5000, 64), (300, 5, 1000, 1),
         (5, 4, 63, 8), (5, 4, 64, 8), (5, 4, 65, 8), (2000, 9, 9000, 3)]


@pytest.mark.parametrize("rows,width,npages,page", SIZES)
@pytest.mark.parametrize("seed", [1, 2])
def test_a_server_s_steps(rows, width, npages, page, seed):
    """All of them in turn, with rows and pairs named twice, outside of the table and in
    conflict."""
    b = Both(rows, width, npages, page, seed, ld=width + 3)
    b.same()
    rng = b.rng
    for step in range(6):
        b.grow(2 * page)
        b.take()
        n = rng.randint(1, max(1, rows // 3))
        b.fork([rng.randint(-1, rows) for _ in range(n)], [rng.randint(-1, rows) for _ in range(n)])
        if step % 2:
            b.compact()
        b.free([rng.randint(-1, rows) for _ in range(max(1, rows // 4))])
    b.compact()


def test_large_pool():
    """More pages than the small notes hold, and the most that a pool may have."""
    for npages in (65536, 65537, 70001, 1 << 20):
        b = Both(500, 100, npages, 4, 3, words=4)
        b.fork([1, 2, 3, 4], [10, 11, 12, 13])
        b.grow(9)
        b.take()
        b.free([5, 6, 7])
        b.compact()


def test_full_pool():
    """No free page: entries stay -1, and the count says how many."""
    b = Both(8, 6, 20, 4, 5, fill=0.0)
    b.ref.len = [24, 24, 24, 5, 0, 1, 4, 30]
    b.len.copy_(ints(b.ref.len))
    b.take()
    b.take()
    b.fork([3, 0, 5], [4, 7, 6])
    b.free([0])
    b.take()
    b.compact()


def test_fork_shares_and_copies():
    b = Both(6, 4, 16, 8, 1, fill=0.0)
    b.ref.len = [20, 16, 0, 0, 0, 0]
    b.len.copy_(ints(b.ref.len))
    b.take()
    b.fork([0, 0, 1], [2, 3, 4])
    assert b.ref.t[2][:2] == b.ref.t[0][:2] and b.ref.t[2][2] not in (b.ref.t[0][2], -1)
    assert b.ref.t[4] == b.ref.t[1] and b.ref.refs[b.ref.t[0][0]] == 3
    b.fork([0], [2])            # again, over its own fork
    b.fork([2], [2])            # itself: left out
    b.fork([0, 2], [2, 5])      # a parent that is a child: left out
    b.fork([], [])
    b.free([0, 0, 0])
    b.free([])
    b.free([2, 3])


def test_nothing_held():
    b = Both(5, 3, 10, 4, 1, fill=0.0)
    b.take()
    b.free([0, 1, 2, 3, 4])
    b.compact()
    b = Both(0, 3, 10, 4, 1)
    b.take()
    b.free([0])
    b.compact()
    b = Both(3, 0, 10, 4, 1)
    b.grow(9)
    b.take()
    b.free([1])
    b.fork([0], [1])
    b.compact()


@pytest.mark.parametrize("words", [4, 8, 1020, 1024, 1028, 4096, 4100, 10240])
def test_copy(words):
    pages = new_pages(40, words)
    want = pages.clone()
    src, dst = [3, 3, -1, 5, 7, 40, 9, 11, 12], [20, 21, 22, -5, 7, 23, 24, 40, 39]
    qig.copy_pages(pages, ints(src), ints(dst))
    for a, b in zip(src, dst):
        if 0 <= a < 40 and 0 <= b < 40:
            want[b] = want[a]
    torch.cuda.synchronize()
    assert torch.equal(pages, want)
    qig.copy_pages(pages, ints([]), ints([]))
    assert torch.equal(pages, want)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float64])
def test_copy_strided_pages(dtype):
    """Pages with something between them, of any type."""
    store = torch.arange(30 * 5 * 32, device="cuda").remainder(100).to(dtype).view(30, 5, 32)
    want = store.clone()
    pages = store[:, 1:4]
    qig.copy_pages(pages, ints([0, 1]), ints([10, 11]))
    want[10:12, 1:4] = want[0:2, 1:4]
    assert torch.equal(store, want)


def test_far_pages():
    """Pages behind 2^32 bytes."""
    pages = torch.zeros((5000, 1 << 20), dtype=torch.uint8, device="cuda")
    pages[4999] = torch.arange(1 << 20, device="cuda").remainder(251).to(torch.uint8)
    qig.copy_pages(pages, ints([4999]), ints([4500]))
    assert torch.equal(pages[4500], pages[4999])
    t, lens, refs = ints([[4999, 4500]]), ints([2]), torch.zeros(5000, dtype=torch.int32, device="cuda")
    refs[[4999, 4500]] = 1
    assert int(qig.compact_pages(pages, t, refs)) == 2
    assert t.tolist() == [[1, 0]] and torch.equal(pages[0], pages[4999]) and torch.equal(pages[1], pages[4999])


def test_captured():
    """A server's step in a graph: replayed on what the pool holds then."""
    b, c = Both(30, 12, 500, 8, 9), Both(30, 12, 500, 8, 9)
    parents, children, rows = ints([1, 2, 5]), ints([7, 8, 9]), ints([3, 4])
    grown = ints([3] * 30)

    def step(x):
        qig.free_pages(x.t, x.len, x.refs, rows)
        m = qig.fork_pages(x.pages, x.t, x.len, x.refs, parents, children, 8)
        x.len.add_(grown)
        n = qig.take_pages(x.t, x.len, x.refs, 8)
        u = qig.compact_pages(x.pages, x.t, x.refs)
        return m, n, u

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    held = [t.clone() for t in (b.t, b.len, b.refs, b.pages)]
    with torch.cuda.stream(side):
        step(b)
    torch.cuda.current_stream().wait_stream(side)
    for t, h in zip((b.t, b.len, b.refs, b.pages), held):
        t.copy_(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(b)
    for t, h in zip((b.t, b.len, b.refs, b.pages), held):
        t.copy_(h)
    for _ in range(4):
        graph.replay()
        want = step(c)
        torch.cuda.synchronize()
        assert [int(x) for x in out] == [int(x) for x in want]
        assert torch.equal(b.t, c.t) and torch.equal(b.len, c.len) and torch.equal(b.refs, c.refs)
        assert torch.equal(b.pages, c.pages)


def test_a_length_beyond_the_table():
    """Takes the entries that the table has; what is beyond it is not missing."""
    t = torch.tensor([[3, 5], [-1, -1], [7, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([33, 1000, 16], dtype=torch.int32, device="cuda")
    refs = torch.zeros(9, dtype=torch.int32, device="cuda")
    refs[[3, 5, 7]] = 1
    assert int(qig.take_pages(t, lens, refs, 16)) == 0
    assert t.tolist() == [[3, 5], [0, 1], [7, -1]] and refs.tolist() == [1, 1, 0, 1, 0, 1, 0, 1, 0]
    refs[:] = 1
    t[1] = -1
    assert int(qig.take_pages(t, lens, refs, 16)) == 2
    assert t.tolist() == [[3, 5], [-1, -1], [7, -1]] and refs.tolist() == [1] * 9
