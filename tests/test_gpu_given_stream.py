"""Results that a call on a given stream allocates: their memory is not in use
by another stream, neither before the call nor after it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SLEEP = 100_000_000   # cycles: some tens of milliseconds


@pytest.fixture(scope="module")
def qig():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as q
    q.load()
    return q


def _calls(qig):
    """name -> call(stream) -> its results.  Outputs of 2 MB and more, each in a
    block of its own."""
    torch.manual_seed(3)
    x = torch.randn(1024, 4096, device="cuda")
    W, sw = qig.quantize_i8(torch.randn(1024, 4096, device="cuda"))
    q, s = qig.quantize_i8(x)
    logits = torch.randn(1 << 18, 8, device="cuda")
    ids, w = qig.route_experts(logits, 2)
    plan = qig.plan_experts(ids[:512].contiguous(), 4)
    We, swe = W.view(4, 256, 4096), sw.view(4, 256)
    h = torch.randn(2048, 1024, device="cuda")
    wt = torch.rand(1024, 2, device="cuda")
    blocks = torch.zeros(4096 * 16 * 144, dtype=torch.uint8, device="cuda")   # q4_K, all scales 0
    q8 = qig.quantize_q8_pad40(x)
    return {
        "quantize_i8": lambda st: qig.quantize_i8(x, stream=st)[:1],
        "mm_i8": lambda st: (qig.mm_i8(W, sw, q, s, stream=st),),
        "route_experts": lambda st: qig.route_experts(logits, 2, stream=st),
        "plan_experts": lambda st: (qig.plan_experts(ids, 8, stream=st),),
        "mm_i8_experts": lambda st: (qig.mm_i8_experts(We, swe, q[:512], s[:512], plan, 1024, stream=st),),
        "combine_experts": lambda st: (qig.combine_experts(h, wt, stream=st),),
        "quantize_q8_pad40": lambda st: (qig.quantize_q8_pad40(x, stream=st),),
        "quantize_q8_tiled": lambda st: (qig.quantize_q8_tiled(x, stream=st),),
        "mmq_q4k": lambda st: (qig.mmq_q4k(blocks, 4096, 4096, q8, 1024, stream=st),),
        "prepare_q4k": lambda st: (qig.prepare_q4k(blocks, 4096, 4096, stream=st),),
    }


NAMES = ["quantize_i8", "mm_i8", "route_experts", "plan_experts", "mm_i8_experts", "combine_experts",
         "quantize_q8_pad40", "quantize_q8_tiled", "mmq_q4k", "prepare_q4k"]


@pytest.mark.parametrize("name", NAMES)
def test_result_of_a_given_stream_is_memory_of_its_own(qig, name):
    call = _calls(qig)[name]
    want = [t.clone() for t in call(None)]
    sizes = [t.untyped_storage().nbytes() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    print(name, sizes, flush=True)
    # blocks of the results' sizes whose last use on the current stream is still to come
    old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(SLEEP)
    for t in old:
        t.fill_(0x7B)
    del old, t
    got = call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), "overwritten by work of the current stream"
    # read late on the current stream, and let go before that read has run
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    late = [t.clone() for t in got]
    del got
    again = call(s)
    with torch.cuda.stream(s):
        for t in again:
            t.fill_(3)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(late, want)), "handed out again before the current stream had read it"
