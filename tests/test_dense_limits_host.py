"""The ends of the dense int8 operators' ranges, refused on the host (no GPU: the
pointers are never dereferenced)."""
import pytest
import torch

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


# --- the binding, on tensors that have a shape and a device but no memory ---------------------------------
class Calls:
    """Stands in for the library: notes its calls, which all succeed."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        def call(*args):
            self.made.append((name, args))
            return 256 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def fake(L, monkeypatch):
    from torch._subclasses.fake_tensor import FakeTensorMode
    calls = Calls()
    monkeypatch.setattr(L, "lib", lambda: calls)
    monkeypatch.setattr(L, "status_string", str)
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda dev: 0)
    L._room_bytes.cache_clear()
    L._backward_bytes.cache_clear()
    with FakeTensorMode():
        yield calls
    L._room_bytes.cache_clear()  # what the stand-in answered is no size
    L._backward_bytes.cache_clear()


def t8(*shape):
    return torch.empty(shape, dtype=torch.int8, device="cuda")


def f32(*shape):
    return torch.empty(shape, device="cuda")


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_binding_refuses_sizes_of_more_than_32_bits(L, fake):
    """The library's sizes are 32-bit: 2^32 + 8 tokens would arrive there as 8."""
    big = (1 << 32) + 8
    for i, call in enumerate([
            lambda: L.quantize_act_token(f32(1, big)),
            lambda: L.int8_matmul(t8(big, 1), f32(big), t8(4, 1), f32(4)),
            lambda: L.int8_matmul(t8(1, big), f32(1), t8(4, big), f32(4)),
            lambda: L.int8_matmul(t8(1, 1), f32(1), t8(big, 1), f32(big)),
            lambda: L.gated_ffn(t8(big, 1), f32(big), t8(4, 1), f32(4), t8(4, 1), f32(4)),
            lambda: L.gated_ffn(t8(1, 1), f32(1), t8(big, 1), f32(big), t8(big, 1), f32(big)),
            lambda: L.int8_matmul_backward(f32(big, 4), None, None, t8(4, 8), f32(4)),
            lambda: L.int8_matmul_backward(f32(4, big), None, None, t8(big, 8), f32(big)),
            lambda: L.int8_matmul_backward(f32(4, 4), None, None, t8(4, big), f32(4)),
            lambda: L.gated_ffn_backward(f32(2, 4), torch.empty((2, 2, 4), dtype=torch.int32, device="cuda"), f32(2),
                                         t8(4, big), f32(4), t8(4, big), f32(4)),
            lambda: L.dense_ffn(f32(big, 4), L.ExpertBank(*(t8(1, 4, 4).view(torch.uint8) for _ in range(3)),
                                                          *(f32(1, 4) for _ in range(3))))]):
        with pytest.raises(L.MoeError) as e:
            call()
        assert e.value.status == EUNSUPPORTED and not fake.made, i


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_quantiser_takes_any_number_of_rows(L, fake):
    q, d = L.quantize_act_token(f32((1 << 32) + 8, 1))
    assert q.shape == ((1 << 32) + 8, 1) and fake.made[0][1][2] == (1 << 32) + 8


@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_backward_workspace_is_sized_for_its_device(L, fake, monkeypatch):
    """The gated backward's workspace grows with the device's SMs: a size asked for one device is not
    taken for another."""
    here = [0]
    monkeypatch.setattr(L, "_current_device", lambda: here[0])
    sent = []

    def answer(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 1000 * (here[0] + 1)
            sent.append(args[-2])  # the workspace's bytes
            return 0
        return call
    monkeypatch.setattr(Calls, "__getattr__", answer)
    for here[0] in (0, 1, 0):
        def on(t):
            return t.to(f"cuda:{here[0]}")
        w, s = on(t8(12, 12)), on(f32(12))
        L.gated_ffn_backward(on(f32(801, 12)), on(torch.empty((2, 801, 12), dtype=torch.int32, device="cuda")),
                             on(f32(801)), w, s, w, s)
    assert sent == [1000, 2000, 1000]
