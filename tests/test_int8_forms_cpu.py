"""Which kernel a product takes, on the CPU: the rule's ranges, and the sizes
that the GPU tests of the forms rely on."""
import pytest

import quant_integer_gemm_amd as qig


@pytest.mark.parametrize("args", [(-1, 8, 16, 4, 0, 0), (513, 8, 16, 4, 0, 0), (0, 0, 16, 4, 0, 0), (0, 8, 0, 4, 0, 0),
                                  (0, 8, 131072, 4, 0, 0), (0, 8, 16, 0, 0, 0), (0, 8, 16, 4, 2, 0),
                                  (0, 1 << 30, 16, 4, 0, 0)])
def test_refuses_sizes_that_the_products_refuse(args):
    assert qig.load().mm_i8_form(*args) == -1


def test_forms_over_the_sizes():
    form = qig.load().mm_i8_form
    assert form(0, 3584, 3584, 1, 0, 1) == 1601
    assert form(0, 3584, 3584, 512, 0, 1) == 6441
    assert form(0, 18944, 3584, 2630, 1, 1) == 25621
    assert form(0, 3584, 18944, 2630, 0, 1) == 19221
    assert form(0, 3584, 18944, 32, 0, 0) == 6441 and form(0, 3584, 18944, 32, 0, 1) == 6444
    # a split needs a workspace and at least 16 steps a share
    assert form(0, 200, 4000, 70, 0, 0) == 6441 and form(0, 200, 4000, 70, 0, 1) == 6442
    assert form(0, 200, 3900, 70, 0, 1) == 6441
    # the few-token kernel's launch ends at 2^27 weight rows
    assert form(0, (1 << 27) - 16, 16, 16, 0, 0) == 1601 and form(0, (1 << 27) + 1, 16, 16, 0, 0) // 100 >= 64
    # experts: by the rows that each has on average
    assert form(64, 2368, 3584, 24, 1, 0) == 3241
    assert form(64, 2368, 3584, 2560, 1, 0) == 12821
    assert form(64, 2368, 3584, 15780, 1, 0) == 25621


def test_sizes_of_the_gpu_tests():
    import test_gpu_int8_forms as t
    form = qig.load().mm_i8_form
    for f, nt, rows in t.DENSE:
        assert all(form(0, rows // (1 + g), i, nt, g, 0) == f for i in t.IDS for g in (0, 1)), (f, nt, rows)
        assert f // 100 == 64 or nt % (f // 100) in (37, 101, 165, 229)
    assert {f for f, _, _ in t.DENSE} == {6421, 19221, 25621}
    for f, nt, k, ne, rows in t.EXPERTS:
        for i in t.IDS:
            r = rows or (25400000 // (ne * i) + 7) // 2 * 2
            assert all(form(ne, r // (1 + g), i, nt * k, g, 0) == f for g in (0, 1)), (f, i)
