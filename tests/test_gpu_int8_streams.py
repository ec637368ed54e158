"""Default workspaces, inside captures too, and streams given by their handles."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

COUNTERS = 16384   # a workspace's last bytes


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


def _split_operands(seed):
    """A product that splits its sums when it has a workspace."""
    torch.manual_seed(seed)
    nt, od, id_ = 70, 200, 8192
    W = torch.randint(-128, 128, (od, id_), dtype=torch.int8, device="cuda")
    q = torch.randint(-127, 128, (nt, id_), dtype=torch.int8, device="cuda")
    return W, torch.rand(od, device="cuda") * 0.02, q, torch.rand(nt, device="cuda") * 1e-3


def test_one_default_workspace_a_capture(qig):
    """The calls of a capture share one workspace, made in it and not known to
    another capture; the graph zeroes its counters alone."""
    a = _split_operands(1)
    dev = a[0].device
    want = qig.mm_i8(*a)
    ys = [torch.zeros_like(want) for _ in range(4)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs, spaces = [], []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            w0 = qig.workspace(dev)
            qig.mm_i8(*a, y=ys[2 * i], ws=w0)
            w1 = qig.workspace(dev)
            qig.mm_i8(*a, y=ys[2 * i + 1], ws=w1)
        assert w0.data_ptr() == w1.data_ptr(), "a second workspace in one capture"
        graphs.append(gr)
        spaces.append(w0)
    assert spaces[0].data_ptr() != spaces[1].data_ptr()
    partial = qig.load().mmq_workspace_bytes() - COUNTERS
    for w in spaces:
        assert w.numel() == partial + COUNTERS
    for i in (1, 0, 0, 1):
        for y in ys:
            y.zero_()
        spaces[i].fill_(0xA5)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[2 * i], want) and torch.equal(ys[2 * i + 1], want), i
        assert int(torch.count_nonzero(spaces[i][partial:])) == 0, "counters"
        assert bool((spaces[i][partial - 4096:partial] == 0xA5).all()), "the partial sums' slots were filled"
        assert torch.equal(qig.mm_i8(*a), want)


def test_new_workspace_has_zero_counters(qig):
    """Also where its memory held something else."""
    n = int(qig.load().mmq_workspace_bytes())
    torch.cuda.empty_cache()
    old = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    del old
    ws = qig.new_workspace("cuda")
    assert ws.numel() == n and ws.dtype == torch.uint8
    assert int(torch.count_nonzero(ws[-COUNTERS:])) == 0
    a = _split_operands(2)
    assert torch.equal(qig.mm_i8(*a), qig.mm_i8(*a, ws=ws))
    assert int(torch.count_nonzero(ws[-COUNTERS:])) == 0


class Handle:
    """A stream of another library: its handle alone."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def test_stream_given_by_its_handle(qig):
    """Whatever has a `cuda_stream` names a stream, for the default workspace
    as for the calls."""
    a = _split_operands(3)
    want = qig.mm_i8(*a)
    x = torch.randn(5, 300, device="cuda")
    q0, s0 = qig.quantize_i8(x)
    y = torch.zeros_like(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    h = Handle(s)
    ws = qig.workspace(a[0].device, h)
    assert ws.data_ptr() == qig.workspace(a[0].device, s).data_ptr()
    qig.mm_i8(*a, y=y, ws=ws, stream=h)
    z = qig.mm_i8(*a, ws=ws, stream=h)
    q1, s1 = qig.quantize_i8(x, stream=h)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want)
    assert torch.equal(q0, q1) and torch.equal(s0, s1)
