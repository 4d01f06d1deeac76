"""Limits of the router's training calls, without a GPU (refused before any HIP call; the pointers are never dereferenced)."""
import ctypes
import os

import pytest

import combine_router_gemm_amd as moe

UNSUPPORTED = -2
P = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.library_path()):
        pytest.skip("HIP library not built (python -m combine_router_gemm_amd.build)")
    return moe.load_library()


@pytest.mark.parametrize("S", [(1 << 30) + 1, (1 << 31) - 2, (1 << 31) - 1])
def test_balance_refuses_sequences_whose_numbers_do_not_add_up_in_31_bits(lib, S):
    """A token's sequence is found by halving [0, S): the sum of two sequence numbers has to stay within an int."""
    assert lib.moe_balance_loss(P, P, P, None, 4, 1, 1, S, 1.0, P, P, P, P, 1 << 62, None) == UNSUPPORTED
