"""The ends of the dense int8 operators' ranges, refused on the host (no GPU: the
pointers are never dereferenced)."""
import pytest

from quantized_routed_expert_group_b200 import build

A = 0x1000
EUNSUPPORTED = -2
LONGEST = (1 << 31) - (1 << 16)  # columns and channels are counted in 32 bits


@pytest.fixture(scope="module")
def L():
    build.build_lib()
    from quantized_routed_expert_group_b200 import moe
    return moe


@pytest.mark.parametrize("cols", [LONGEST + 1, (1 << 31) - 4095, (1 << 31) - 1])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_quantise_refuses_rows_past_its_column_index(L, cols, dtype):
    """A thread's column index steps past the row's end by up to 512 x 8: near 2^31 it would turn
    negative, and the loop would go on in front of the row."""
    assert L.lib().moe_quantize_act_token(A, dtype, 1, cols, cols, A, cols, A, None) == EUNSUPPORTED


TOO_LONG = [LONGEST + 1, (1 << 31) - 100, (1 << 31) - 1]


@pytest.mark.parametrize("n", TOO_LONG)
def test_products_refuse_channels_past_their_index(L, n):
    """A tile's last channel index is up to 255 past the last channel: near 2^31 it would turn negative
    and pass for one in front of the row."""
    lib = L.lib()
    assert lib.moe_int8_matmul(A, 64, A, 17, A, 64, A, n, 64, None, A, 1, n, None, None, 0, None) == EUNSUPPORTED
    assert lib.moe_gated_ffn(A, 64, A, 17, A, 64, A, A, 64, A, n, 64, 0, A, 1, n, None, None, 0, None) == EUNSUPPORTED
    assert lib.moe_int8_matmul_backward(A, 1, 32, A, A, 4, A, n, A, 32, n, A, n, A, A, A, 1 << 62, None) == EUNSUPPORTED
    assert lib.moe_gated_ffn_backward(A, 1, 32, A, A, 4, A, n, A, A, n, A, 32, n, 0, A, n, A, A, A, 1 << 62,
                                      None) == EUNSUPPORTED
    assert lib.moe_int8_forward_workspace_bytes(1, 17, n, 1001) == 0
    assert lib.moe_int8_backward_workspace_bytes(1, 17, 32, n, 1) == 0


def test_products_still_take_the_longest(L):
    """Sizes in range pass the checks: their workspace is given."""
    assert L.lib().moe_int8_forward_workspace_bytes(1, 17, LONGEST, 1001) > LONGEST * 1001
    assert L.lib().moe_int8_backward_workspace_bytes(1, 17, 32, LONGEST, 1) > 0
