"""Sizes of the attention operators at the end of 32 bits, without a GPU."""
import pytest

from test_attend_cpu import BIG, PACKED, _packed, _prompt


@pytest.mark.parametrize("nk", [BIG - 1, BIG - 64, BIG - 257, BIG - 1023])
def test_keys_that_a_kernels_steps_would_pass(nk):
    """attend_prompt counts keys in ints, up to 256 at a step and one step ahead: with more keys
    than 2^31 - 1024 the last steps would wrap, and read behind the tensors' beginning."""
    assert _prompt(nt=0, nk=nk) == -1 and _prompt(nseq=0, nk=nk) == -1
    assert _packed(0, PACKED[0], _11=nk) == -1
    assert _prompt(nt=0, nk=BIG - 1024) == 0 and _packed(0, PACKED[0], _11=BIG - 1024) == 0
