"""What the dense int8 operators do with tensors that require a gradient: they record
none, so they refuse them where one would be recorded (no GPU: a stand-in for the
library, tensors without memory)."""
import pytest
import torch

from test_dense_limits_host import L, f32, fake, t8  # noqa: F401

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer")


def i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def bank(L, leaf=None):
    parts = [t8(1, 8, 4).view(torch.uint8), t8(1, 8, 4).view(torch.uint8), t8(1, 4, 8).view(torch.uint8),
             f32(1, 8), f32(1, 8), f32(1, 4)]
    if leaf is not None:
        parts[leaf].requires_grad_()
    return L.ExpertBank(*parts)


def leaf(*shape):
    return f32(*shape).requires_grad_()


CALLS = {
    "x of the quantiser": lambda L, f: L.quantize_act_token(f(2, 4)),
    "xd": lambda L, f: L.int8_matmul(t8(2, 4), f(2), t8(8, 4), f32(8)),
    "s": lambda L, f: L.int8_matmul(t8(2, 4), f32(2), t8(8, 4), f(8)),
    "bias": lambda L, f: L.int8_matmul(t8(2, 4), f32(2), t8(8, 4), f32(8), bias=f(8)),
    "out": lambda L, f: L.int8_matmul(t8(2, 4), f32(2), t8(8, 4), f32(8), out=f(2, 8)),
    "s_gate": lambda L, f: L.gated_ffn(t8(2, 4), f32(2), t8(8, 4), f(8), t8(8, 4), f32(8)),
    "s_up": lambda L, f: L.gated_ffn(t8(2, 4), f32(2), t8(8, 4), f32(8), t8(8, 4), f(8)),
    "dy": lambda L, f: L.int8_matmul_backward(f(2, 8), None, None, t8(8, 4), f32(8)),
    "s of the backward": lambda L, f: L.int8_matmul_backward(f32(2, 8), i32(2, 8), f32(2), t8(8, 4), f(8)),
    "dh": lambda L, f: L.gated_ffn_backward(f(2, 8), i32(2, 2, 8), f32(2), t8(8, 4), f32(8), t8(8, 4), f32(8)),
    "x of the feed-forward": lambda L, f: L.dense_ffn(f(2, 4), bank(L)),
    "scales of a bank": lambda L, f: L.dense_ffn(f32(2, 4), bank(L, None if f is f32 else 4)),
}


@pytest.mark.parametrize("name", CALLS)
def test_leaves_are_refused_where_a_gradient_would_be_recorded(L, fake, name):
    call = CALLS[name]
    with pytest.raises(ValueError, match="gradient"):
        call(L, leaf)
    assert not fake.made
    with torch.no_grad():  # as inside a torch.autograd.Function
        call(L, leaf)
    assert fake.made
    call(L, f32)
