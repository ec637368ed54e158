"""Launches of 2^32 and more threads are refused before they reach the GPU
(the runtime would run a part of them without an error)."""
import ctypes

import pytest

import quant_integer_gemm_amd as qig

P = ctypes.c_void_p(0x10000)   # never dereferenced: the calls are refused


def test_products_with_more_tiles_than_a_launch_holds():
    lib = qig.load()
    od = (1 << 30) - 1
    # 65 tokens: two 64-row tiles of 2^23 (gated: 2^24) columns, 256 threads each
    assert lib.mm_i8(P, 16, P, od, 16, P, 16, P, 65, None, 0, P, 0, od, None, None) == -1
    assert lib.mm_i8(P, 16, P, od, 16, P, 16, P, 65, None, 1, P, 1, od, None, None) == -1
    # 1026 rows of 512 experts: 32-row tiles, up to 545 of them
    assert lib.mm_i8_experts(P, 16, P, 512, 1 << 25, 16, P, 16, P, 1026, 1, P, None, 0, P, 0, 1 << 25, None) == -1


def test_k_quant_calls_too():
    lib = qig.load()
    # a thread for four elements; eight workgroups of 256 for each of 2^21 records
    assert lib.quantize_q8_pad40(P, 1 << 22, 4096, 4096, P, None) == -1
    assert lib.quantize_q8_tiled(P, 1 << 22, 8192, 8192, P, None) == -1
    # 64 x 64 tiles of 256 threads
    assert lib.mmq_q4k(P, 1 << 20, 256, P, 1 << 16, P, 1 << 20, None) == -1


def test_experts_without_weight_rows_pass_the_stride_check():
    """Four experts of no rows have no stride to get wrong: on the CPU the call
    ends at its check of the device."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(qig.QigError, match="GPU tensor"):
        qig.mm_i8_experts(z(4, 0, 32, dtype=torch.int8), z(4, 0), z(3, 32, dtype=torch.int8), z(3),
                          z(12, dtype=torch.int32), 6)
