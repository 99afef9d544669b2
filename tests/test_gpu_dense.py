"""The dense int8 operators on the GPU against their formulas in 64 bits
(bounds derived in dense_helpers.py).  Integer sums and codes are exact."""
import numpy as np
import pytest
import torch

import dense_helpers as dh
from quantized_routed_expert_group_b200 import moe

pytestmark = pytest.mark.gpu

DT = dh.DTYPES
# tokens, cols, rows: one of everything, sizes around the tiles (16, 32, 64, 128 tokens, 128 rows, 128 codes),
# odd ones whose rows are no multiple of 16, 8 or 4 bytes, long rows
SIZES = [(24, 1040, 300), (32, 272, 65), (20, 999, 77), (1, 1, 1), (1, 16, 1), (1, 6144, 300), (2, 127, 5), (3, 129, 130), (4, 512, 128), (5, 2048, 257),
         (16, 1000, 77), (17, 128, 384), (33, 100, 64), (64, 1040, 129), (65, 36, 127), (128, 256, 128),
         (129, 260, 131), (300, 1000, 500), (257, 1536, 640)]
LARGE = [(333, 1001, 777), (640, 1003, 1501), (700, 2048, 1504), (1030, 1024, 528), (513, 272, 1032), (256, 16, 16), (2500, 128, 4000), (4000, 1040, 3120), (40, 64, 6200), (30, 48, 7001), (21, 32, 16500), (600, 64, 8192), (1500, 64, 40), (3000, 48, 333)]


def cuda(*ts):
    return [t.cuda() for t in ts]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K", [(1, 1), (1, 6144), (3, 33), (5, 1000), (64, 2048), (7, 4104), (2, 20000), (2, 70001)])
def test_quantize_token(T, K, dtype):
    gen = torch.Generator().manual_seed(T * 7 + K)
    x = torch.randn((T, K), generator=gen) * torch.exp(2 * torch.randn((T, 1), generator=gen))
    if K > 8:
        x[0, :8] = torch.tensor([0.5, -0.5, 1.5, -1.5, 2.5, -2.5, 63.5, 127.0])  # ties: the scale is 1
        x[0, 8:] = 0
    if T > 2:
        x[1] = 0
        x[2] = 1e-36 if dtype != "fp16" else 0.0
    x = x.to(DT[dtype])
    q, d = moe.quantize_act_token(x.cuda())
    xn = x.float().numpy()
    amax = np.abs(xn).max(1)
    live = amax >= np.float32(2.0 ** -112)
    want_d = np.where(live, amax / np.float32(127), np.float32(0)).astype(np.float32)
    inv = np.where(live, np.float32(1) / np.where(live, want_d, np.float32(1)), np.float32(0)).astype(np.float32)
    v = (xn * inv[:, None]).astype(np.float32)
    want_q = np.clip(np.sign(v) * np.floor(np.abs(v).astype(np.float64) + 0.5), -127, 127).astype(np.int8)
    np.testing.assert_array_equal(d.cpu().numpy().view(np.uint32), want_d.view(np.uint32))
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


def test_quantize_token_non_finite_rows():
    x = torch.randn(5, 100)
    x[1, 3], x[2, 99], x[3, 0] = float("nan"), float("inf"), float("-inf")
    q, d = moe.quantize_act_token(x.cuda())
    assert torch.isnan(d.cpu()).tolist() == [False, True, True, True, False]
    assert not q[1:4].any() and q[0].any() and q[4].any()
    y = moe.int8_matmul(q, d, torch.ones((3, 100), dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"))
    assert torch.isnan(y.cpu()).all(1).tolist() == [False, True, True, True, False]


@pytest.mark.parametrize("T,K,N", SIZES + LARGE)
@pytest.mark.parametrize("dtype", list(DT))
def test_matmul(T, K, N, dtype):
    x, xd, (w,), (s,), bias, _ = dh.inputs(T + K + N, T, K, N, 1, DT[dtype])
    acc, y, tol = dh.ref_matmul(x, xd, w, s, bias, DT[dtype])
    got, got_acc = moe.int8_matmul(*cuda(x, xd, w, s, bias), out_dtype=DT[dtype], save=True)
    assert torch.equal(got_acc.cpu().double(), acc)
    dh.check("y", got, y, tol)
    _, y, tol = dh.ref_matmul(x, xd, w, s, None, DT[dtype])
    dh.check("y without bias", moe.int8_matmul(*cuda(x, xd, w.view(torch.uint8), s), out_dtype=DT[dtype]), y, tol)
    assert moe.dense_device_error() == 0


@pytest.mark.parametrize("T,K,N", SIZES + LARGE)
@pytest.mark.parametrize("act,dtype", [("silu", "fp32"), ("silu", "bf16"), ("gelu", "fp32"), ("gelu", "fp16")])
def test_gated(T, K, N, act, dtype):
    x, xd, ws, ss, _, _ = dh.inputs(T + K + N, T, K, N, 2, DT[dtype])
    acc, h, tol = dh.ref_gated(x, xd, ws, ss, act, DT[dtype])
    got, got_acc = moe.gated_ffn(*cuda(x, xd, ws[0], ss[0], ws[1], ss[1]), act=act, out_dtype=DT[dtype], save=True)
    assert torch.equal(got_acc.cpu().double(), acc)
    dh.check("h", got, h, tol)
    again = moe.gated_ffn(*cuda(x, xd, ws[0], ss[0], ws[1], ss[1]), act=act, out_dtype=DT[dtype])
    assert torch.equal(got, again)
    assert moe.dense_device_error() == 0


@pytest.mark.parametrize("T,K,N", SIZES + LARGE)
@pytest.mark.parametrize("dtype", list(DT))
def test_matmul_backward(T, K, N, dtype):
    x, xd, (w,), (s,), _, dy = dh.inputs(T + K + N, T, K, N, 1, DT[dtype])
    acc = dh.sums64(x, w)
    refs = dh.ref_matmul_backward(dy, acc, xd, w, s, DT[dtype])
    c = cuda(dy, acc.int(), xd, w, s)
    got = moe.int8_matmul_backward(*c, bias_grad=True)
    for name, g, (want, tol) in zip(("dx", "ds", "dbias"), got, refs):
        dh.check(name, g, want, tol)
    dx, ds, db = moe.int8_matmul_backward(c[0], None, None, c[3], c[4])
    assert ds is None and db is None and torch.equal(dx, got[0])
    assert moe.dense_device_error() == 0


@pytest.mark.parametrize("T,K,N", SIZES + LARGE)
@pytest.mark.parametrize("act,dtype", [("silu", "fp32"), ("silu", "bf16"), ("gelu", "fp32"), ("gelu", "fp16")])
def test_gated_backward(T, K, N, act, dtype):
    x, xd, ws, ss, _, dy = dh.inputs(T + K + N, T, K, N, 2, DT[dtype])
    acc = torch.stack([dh.sums64(x, w) for w in ws])
    refs = dh.ref_gated_backward(dy, acc, xd, ws, ss, act, DT[dtype])
    got = moe.gated_ffn_backward(*cuda(dy, acc.int(), xd, ws[0], ss[0], ws[1], ss[1]), act=act)
    for name, g, (want, tol) in zip(("dx", "ds_gate", "ds_up"), got, refs):
        dh.check(name, g, want, tol)
    assert moe.dense_device_error() == 0


def bank_of(ws, ss):
    g, u, d = (w.view(torch.uint8).cuda()[None] for w in ws)
    sg, su, sd = (s.cuda()[None] for s in ss)
    return moe.ExpertBank(g, u, d, sg, su, sd)


def ffn_inputs(T, H, I, dtype):
    gen = torch.Generator().manual_seed(T + H + I)
    x = torch.randn((T, H), generator=gen).to(DT[dtype])
    ws = [dh.codes(gen, r, c) for r, c in ((I, H), (I, H), (H, I))]
    ss = [(torch.rand(r, generator=gen) + 0.5) / (50.0 * c ** 0.5) for r, c in ((I, H), (I, H), (H, I))]
    return x, ws, ss


# (300, ..) and up run the tiled kernels, up to 32 the weight stream with tokens quantised inside, and
# 1000 x 500 and 36 x 20 rows off the 16-byte grid
FFN = [(1, 256, 128), (1, 6144, 2048), (3, 512, 96), (4, 6144, 2048), (5, 1000, 500), (8, 1024, 304), (9, 1024, 304),
       (16, 2048, 640), (17, 512, 256), (25, 1024, 208), (32, 512, 272), (2, 36, 20), (300, 1024, 512), (130, 264, 72)]


@pytest.mark.parametrize("T,H,I", FFN)
@pytest.mark.parametrize("act,dtype", [("silu", "bf16"), ("gelu", "fp32"), ("silu", "fp16")])
def test_dense_ffn_is_its_steps(T, H, I, act, dtype):
    """The run of the operators equals them called one by one, bit for bit."""
    x, ws, ss = ffn_inputs(T, H, I, dtype)
    bank = bank_of(ws, ss)
    xc = x.cuda()
    got = moe.dense_ffn(xc, bank, act=act)
    q, d = moe.quantize_act_token(xc)
    h = moe.gated_ffn(q, d, bank.w_gate[0], bank.s_gate[0], bank.w_up[0], bank.s_up[0], act=act)
    hq, hd = moe.quantize_act_token(h)
    want = moe.int8_matmul(hq, hd, bank.w_down[0], bank.s_down[0], out_dtype=DT[dtype])
    assert torch.equal(got, want)
    assert moe.dense_device_error() == 0


def strided(t, offset, pitch, fill=None):
    """t as a view of a larger buffer: `offset` elements into it, rows `pitch` elements apart."""
    rows, cols = t.shape
    buf = torch.full((offset + rows * pitch + 64,), 77 if fill is None else fill, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_(t)
    return buf, v


# every loader (16, 8, 4 bytes and single ones), each with short and long batches; row strides beyond the row
@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("offset,extra", [(0, 16), (16, 32), (8, 8), (4, 12), (1, 3), (3, 0), (2, 6)])
def test_strided_operands_and_results(T, offset, extra):
    K, N, dtype = 272, 136, torch.bfloat16
    x, xd, ws, ss, bias, dy = dh.inputs(T + offset, T, K, N, 2, dtype)
    cd = cuda(xd, ss[0], ss[1], bias)
    _, xv = strided(x, offset, K + extra)
    wv = [strided(w, offset, K + extra)[1] for w in ws]
    obuf, ov = strided(torch.zeros((T, N), dtype=dtype), offset, N + extra)
    acc, y, tol = dh.ref_matmul(x, xd, ws[0], ss[0], bias, dtype)
    got = moe.int8_matmul(xv, cd[0], wv[0], cd[1], bias=cd[3], out_dtype=dtype, out=ov)
    assert got is ov
    dh.check("y", ov, y, tol)
    padded = obuf[offset:offset + T * (N + extra)].view(T, N + extra)[:, N:]
    assert (padded == 77).all() and (obuf[:offset] == 77).all() and (obuf[offset + T * (N + extra):] == 77).all()
    sums, h, tol = dh.ref_gated(x, xd, ws, ss, "silu", dtype)
    obuf, ov = strided(torch.zeros((T, N), dtype=dtype), offset, N + extra)
    _, got_acc = moe.gated_ffn(xv, cd[0], wv[0], cd[1], wv[1], cd[2], out_dtype=dtype, out=ov, save=True)
    dh.check("h", ov, h, tol)
    assert torch.equal(got_acc.cpu().double(), sums)
    padded = obuf[offset:offset + T * (N + extra)].view(T, N + extra)[:, N:]
    assert (padded == 77).all() and (obuf[:offset] == 77).all()
    _, dyv = strided(dy, offset, N + extra)
    for name, g, (want, tol) in zip(("dx", "ds_gate", "ds_up"),
                                    moe.gated_ffn_backward(dyv, got_acc, cd[0], wv[0], cd[1], wv[1], cd[2]),
                                    dh.ref_gated_backward(dy, sums, xd, ws, ss, "silu", dtype)):
        dh.check(name, g, want, tol)
    for name, g, (want, tol) in zip(("dx", "ds", "dbias"),
                                    moe.int8_matmul_backward(dyv, got_acc[0].contiguous(), cd[0], wv[0], cd[1], True),
                                    dh.ref_matmul_backward(dy, sums[0], xd, ws[0], ss[0], dtype)):
        dh.check(name, g, want, tol)
    xf = torch.randn((T, K)).to(dtype)
    _, xfv = strided(xf, offset, K + extra)
    (q, d), (q0, d0) = moe.quantize_act_token(xfv), moe.quantize_act_token(xf.cuda())
    assert torch.equal(q, q0) and torch.equal(d, d0)
    assert moe.dense_device_error() == 0


@pytest.mark.parametrize("T,K,N", [(333, 1001, 777), (40, 4093, 1333), (300, 2050, 2809), (700, 3001, 1030),
                                   (129, 8185, 8200), (17, 70001, 33)])
def test_odd_rows_copied_or_as_they_lie(T, K, N):
    """Rows of an odd length give the bits of the same rows at a stride of 16 bytes, with the
    workspace that holds their copies, without one and with one that is too small."""
    gen = torch.Generator().manual_seed(T + K + N)
    xq = torch.randint(-127, 128, (T, K), generator=gen, dtype=torch.int8)
    ws = [torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8) for _ in range(2)]
    xd, *ss = cuda(torch.rand(T, generator=gen), *(torch.rand(N, generator=gen) * 1e-3 for _ in range(2)))
    dy = torch.randn((T, N), generator=gen).cuda()
    pitch = (K + 15) // 16 * 16
    even = [strided(t, 0, pitch, 99)[1] for t in (xq, *ws)]
    odd = cuda(xq, *ws)

    def run(x, wg, wu):
        y, acc = moe.int8_matmul(x, xd, wg, ss[0], out_dtype=torch.bfloat16, save=True)
        h, acc2 = moe.gated_ffn(x, xd, wg, ss[0], wu, ss[1], out_dtype=torch.float32, save=True)
        dx, ds = moe.int8_matmul_backward(dy, acc, xd, wg, ss[0])[:2]
        back = moe.gated_ffn_backward(dy.bfloat16(), acc2, xd, wg, ss[0], wu, ss[1])
        return [y, acc, h, acc2, dx, ds, *back]

    want = run(*even)
    for i, (a, b) in enumerate(zip(run(*odd), want)):
        assert torch.equal(a, b), i
    lib, stream = moe.lib(), torch.cuda.current_stream().cuda_stream
    need = lib.moe_int8_forward_workspace_bytes(2, T, N, K)
    room = torch.empty(need, dtype=torch.uint8, device="cuda")
    for ptr, size in ((None, 0), (room.data_ptr(), need - 1), (room.data_ptr(), need)):
        y, h = torch.empty_like(want[0]), torch.empty_like(want[2])
        assert lib.moe_int8_matmul(odd[0].data_ptr(), K, xd.data_ptr(), T, odd[1].data_ptr(), K, ss[0].data_ptr(), N,
                                   K, None, y.data_ptr(), 1, N, None, ptr, size, stream) == 0
        assert lib.moe_gated_ffn(odd[0].data_ptr(), K, xd.data_ptr(), T, odd[1].data_ptr(), K, ss[0].data_ptr(),
                                 odd[2].data_ptr(), K, ss[1].data_ptr(), N, K, 0, h.data_ptr(), 0, N, None, ptr, size,
                                 stream) == 0
        assert torch.equal(y, want[0]) and torch.equal(h, want[2])
