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
