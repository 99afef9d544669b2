"""Refusals of the dense int8 operators on the host (no GPU: the pointers are
never dereferenced) and what the binding checks."""
import ctypes

import pytest
import torch

from quantized_routed_expert_group_b200 import build

A = 0x1000
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    build.build_lib()
    from quantized_routed_expert_group_b200 import moe
    return moe


MATMUL = dict(xq=A, ldx=64, xd=A, T=4, w=A, ldw=64, s=A, rows=32, cols=64, bias=None, out=A, dtype=0, ldo=32,
              acc=None, ws=None, ws_bytes=0)
GATED = dict(xq=A, ldx=64, xd=A, T=4, wg=A, ldg=64, sg=A, wu=A, ldu=64, su=A, rows=32, cols=64, act=0, out=A,
             dtype=0, ldo=32, acc=None, ws=None, ws_bytes=0)
MATMUL_B = dict(dy=A, dtype=0, lddy=32, acc=A, xd=A, T=4, w=A, ldw=64, s=A, rows=32, cols=64, dx=A, lddx=64, ds=A,
                dbias=A, ws=A, ws_bytes=1 << 30)
GATED_B = dict(dh=A, dtype=0, lddh=32, acc=A, xd=A, T=4, wg=A, ldg=64, sg=A, wu=A, ldu=64, su=A, rows=32, cols=64,
               act=0, dx=A, lddx=64, dsg=A, dsu=A, ws=A, ws_bytes=1 << 30)


@pytest.mark.parametrize("name,base,bad,status", [
    ("moe_int8_matmul", MATMUL, dict(T=-1), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(rows=0), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(cols=0), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(dtype=3), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(xq=None), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(xd=None), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(xd=A + 2), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(w=None), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(s=None), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(out=None), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(out=A + 2), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(out=A + 1, dtype=1), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(ldx=63), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(ldw=63), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(ldo=31), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(bias=A + 1), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(acc=A + 2), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(ws=A + 16), EINVAL),
    ("moe_gated_ffn", GATED, dict(ws=A + 128, ws_bytes=64), EINVAL),
    ("moe_int8_matmul", MATMUL, dict(cols=131072, ldx=131072, ldw=131072), EUNSUPPORTED),
    ("moe_int8_matmul", MATMUL, dict(T=(1 << 28) + 1), EUNSUPPORTED),
    ("moe_int8_matmul", MATMUL, dict(T=0, xq=None, out=None, xd=None), 0),
    ("moe_int8_matmul", MATMUL, dict(T=0, w=None), EINVAL),
    ("moe_gated_ffn", GATED, dict(act=2), EINVAL),
    ("moe_gated_ffn", GATED, dict(wu=None), EINVAL),
    ("moe_gated_ffn", GATED, dict(su=A + 1), EINVAL),
    ("moe_gated_ffn", GATED, dict(ldu=63), EINVAL),
    ("moe_gated_ffn", GATED, dict(ldg=63), EINVAL),
    ("moe_gated_ffn", GATED, dict(ldo=31), EINVAL),
    ("moe_gated_ffn", GATED, dict(cols=131072, ldx=131072, ldg=131072, ldu=131072), EUNSUPPORTED),
    ("moe_gated_ffn", GATED, dict(T=0, xq=None, out=None), 0),
    ("moe_int8_matmul_backward", MATMUL_B, dict(dy=None), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(dx=None), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(acc=None), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(xd=None), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(lddy=31), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(lddx=63), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(ws=None), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(ws=A + 16), EINVAL),
    ("moe_int8_matmul_backward", MATMUL_B, dict(ws_bytes=100), EWORKSPACE),
    ("moe_int8_matmul_backward", MATMUL_B, dict(rows=131072, lddy=131072), EUNSUPPORTED),
    ("moe_gated_ffn_backward", GATED_B, dict(acc=None), EINVAL),
    ("moe_gated_ffn_backward", GATED_B, dict(xd=None), EINVAL),
    ("moe_gated_ffn_backward", GATED_B, dict(act=-1), EINVAL),
    ("moe_gated_ffn_backward", GATED_B, dict(dtype=-1), EINVAL),
    ("moe_gated_ffn_backward", GATED_B, dict(ldu=63), EINVAL),
    ("moe_gated_ffn_backward", GATED_B, dict(ws_bytes=100), EWORKSPACE),
    ("moe_gated_ffn_backward", GATED_B, dict(rows=65536, lddh=65536), EUNSUPPORTED),
])
def test_refusals(L, name, base, bad, status):
    args = dict(base, **bad)
    assert getattr(L.lib(), name)(*args.values(), None) == status


def test_quantize_refusals(L):
    f = L.lib().moe_quantize_act_token
    good = dict(x=A, dtype=0, n=4, cols=64, ldx=64, q=A, ldq=64, d=A)
    for bad in (dict(x=None), dict(x=A + 2), dict(dtype=3), dict(n=-1), dict(cols=0), dict(ldx=63), dict(q=None),
                dict(ldq=63), dict(d=None), dict(d=A + 1)):
        assert f(*dict(good, **bad).values(), None) == EINVAL, bad
    assert f(*dict(good, n=0, x=None).values(), None) == 0


def test_ffn_refusals(L):
    f = L.lib().moe_dense_ffn
    ex = L.MoeExperts(*([A] * 6))
    need = L.lib().moe_dense_ffn_workspace_bytes(4, 64, 32)
    good = dict(x=A, dtype=1, ldx=64, T=4, hidden=64, inter=32, ex=ctypes.byref(ex), act=0, out=A, ldo=64, ws=A,
                ws_bytes=need)
    for bad, status in ((dict(x=None), EINVAL), (dict(act=9), EINVAL), (dict(ldx=63), EINVAL), (dict(ldo=63), EINVAL),
                        (dict(ex=None), EINVAL), (dict(ws=None), EINVAL), (dict(ws=A + 8), EINVAL),
                        (dict(ws_bytes=need - 1), EWORKSPACE), (dict(hidden=0), EINVAL), (dict(T=-1), EINVAL),
                        (dict(ex=ctypes.byref(L.MoeExperts(A, A, None, A, A, A))), EINVAL),
                        (dict(hidden=131072, ldx=131072, ldo=131072), EUNSUPPORTED), (dict(T=0, x=None), 0)):
        assert f(*dict(good, **bad).values(), None) == status, bad


def test_workspace_sizes(L):
    lib = L.lib()
    for n_mats, dtype, planes in ((1, 0, 3), (2, 0, 3), (1, 1, 2), (2, 2, 2)):
        n = lib.moe_int8_backward_workspace_bytes(n_mats, 300, 500, 64, dtype)
        assert n >= planes * 300 * n_mats * 512 + 300 * 8  # planes and row scales
    assert lib.moe_int8_backward_workspace_bytes(1, 0, 8, 64, 0) > 0
    for bad in ((0, 4, 8, 64, 0), (3, 4, 8, 64, 0), (1, -1, 8, 64, 0), (1, 4, 0, 64, 0), (1, 4, 8, 64, 5),
                (2, 4, 65536, 64, 0), (1, 4, 8, 0, 0)):
        assert lib.moe_int8_backward_workspace_bytes(*bad) == 0
    # room for rows off the 16-byte grid, where copying them pays
    room = lib.moe_int8_forward_workspace_bytes
    assert room(1, 300, 3000, 1000) >= 3300 * 1008 and room(2, 300, 3000, 1000) >= 6300 * 1008
    assert room(1, 300, 3000, 1008) == room(1, 16, 3000, 1000) == room(1, 300, 100, 100) == 0
    assert room(0, 300, 3000, 1000) == room(1, 300, 3000, 131072) == room(1, -1, 3000, 1000) == 0
    assert lib.moe_int8_backward_workspace_bytes(1, 4, 3000, 1000, 0) >= 3000 * 1008
    assert lib.moe_dense_ffn_workspace_bytes(4, 64, 32) >= 4 * (64 + 32 + 4 * 32 + 8)
    assert lib.moe_dense_ffn_workspace_bytes(-1, 64, 32) == 0
    assert lib.moe_dense_device_error(None, None) == EINVAL


def test_binding_refuses_host_tensors_and_other_types(L):
    x, v = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="xq"):
        L.int8_matmul(x, v, x, v)
    with pytest.raises(ValueError, match="xq"):
        L.gated_ffn(x, v, x, v, x, v)
    with pytest.raises(ValueError, match="dy"):
        L.int8_matmul_backward(torch.zeros((4, 4)), None, None, x, v)
    with pytest.raises(ValueError, match="dh"):
        L.gated_ffn_backward(torch.zeros((4, 4)), None, v, x, v, x, v)
    with pytest.raises(ValueError, match="x must"):
        L.quantize_act_token(torch.zeros((4, 64), dtype=torch.float64))
    with pytest.raises(ValueError, match="x must"):
        L.dense_ffn(torch.zeros((4, 64)), None)
