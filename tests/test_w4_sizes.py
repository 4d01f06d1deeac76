"""Sizes of the 4-bit and few-token calls at the ends of their arguments' range, without a GPU: exact where the call takes
the sizes, 0 where it refuses them, never a size that has wrapped around."""
import pytest

import combine_router_gemm_amd as moe

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("K", [32, 128, 7168, 2 ** 30, INT_MAX - 511 - 32, INT_MAX - 31, INT_MAX - 63])
@pytest.mark.parametrize("rows", [16, 48, 2 ** 31, 2 ** 36, 2 ** 52, 2 ** 60, 2 ** 63 - 16])
def test_packed_sizes(rows, K):
    takes = K <= INT_MAX - 512 and rows <= (2 ** 63 - 1) // 4 // K  # else moe_quantize_w4 is MOE_ERR_UNSUPPORTED
    assert moe.moe_w4_codes_bytes(rows, K) == (rows // 16 * -(-K // 128) * 1024 if takes else 0)
    assert moe.moe_w4_scales_bytes(rows, K) == (rows // 16 * -(-K // 512) * 256 if takes else 0)
    assert moe.load_library().moe_quantize_w4(None, moe.MOE_BF16, rows, K, None, None, None) == (-1 if takes else -2)


def test_layer_workspace():
    size = moe.moe_layer_decode_workspace_bytes
    # h in two parts or fp32, x in the matrix step's order
    for H, F in ((2 ** 23, 2 ** 20), (64, 2 ** 20), (2 ** 23, 32)):
        assert size(32, H, 8, 8, F, moe.MOE_BF16) >= 32 * 8 * F * 4 + 32 * H * 2
    for H, F in ((2 ** 23 + 8, 64), (64, 2 ** 20 + 8), (INT_MAX, 64), (64, INT_MAX), (INT_MAX, INT_MAX)):
        assert size(32, H, 8, 8, F, moe.MOE_BF16) == 0


def test_mlp_workspace():
    size = moe.moe_expert_mlp_w4_workspace_bytes
    for T, F in ((1 << 16, 2048), (1, 1 << 25)):
        assert size(T, 1, 8, 1, T, F) >= T * F * 4
    # F 2^26: the scales of 2 F rows take 2^27 / 16 * 256 = 2^31 bytes for the smallest H, past 31 bits
    for T, k, C, F in ((1, 1, 1, 1 << 26), (1, 1, 1, 1 << 29), (1, 1, 1, INT_MAX), (INT_MAX, 8, INT_MAX, INT_MAX),
                       (INT_MAX, INT_MAX, INT_MAX, INT_MAX), (1 << 20, 8, 1 << 20, 1 << 12)):
        assert size(T, k, 8, 1, C, F) == 0
