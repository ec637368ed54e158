"""Experts without outputs: the calls have nothing to do and say so."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("ne", [1, 4])
@pytest.mark.parametrize("glu", [False, True])
def test_experts_without_weight_rows(ne, glu):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quant_integer_gemm_amd as qig
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    plan = qig.plan_experts(ids, ne)
    q, s = qig.quantize_i8(torch.ones(3, 32, device="cuda"))
    W = torch.zeros((ne, 0, 32), dtype=torch.int8, device="cuda")
    y = qig.mm_i8_experts(W, torch.zeros(ne, 0, device="cuda"), q, s, plan, 6, glu=glu)
    assert y.shape == (6, 0)
    assert qig.combine_experts(y, torch.ones(3, 2, device="cuda")).shape == (3, 0)
    torch.cuda.synchronize()
