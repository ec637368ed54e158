"""Default workspaces, and streams given by their handles."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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
