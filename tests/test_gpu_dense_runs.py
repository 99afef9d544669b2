"""The dense int8 operators as a program runs them: together in a training step,
on other streams, captured into graphs, at the ends of their ranges, and with
rows that hold nothing or too much."""
import math

import pytest
import torch

import dense_helpers as dh
from quantized_routed_expert_group_b200 import moe

pytestmark = pytest.mark.gpu

DT = dh.DTYPES


def packed(gen, rows, cols):
    """A weight as the framework packs it (int8 rows with a scale each), and its codes."""
    w = torch.randn((rows, cols), generator=gen) * 0.02
    p, s = moe.pack_weights(w.cuda(), 8)
    return p, s, p.view(torch.int8).cpu()


class Ffn:
    """A dense feed-forward of the operators with its backward pass, the codes
    constant and the quantisers passing gradients through."""

    def __init__(self, gen, H, I):
        (self.wg, self.sg, self.qg), (self.wu, self.su, self.qu), (self.wd, self.sd, self.qd) = (
            packed(gen, I, H), packed(gen, I, H), packed(gen, H, I))

    def forward(self, x):
        q, d = moe.quantize_act_token(x)
        h, acc = moe.gated_ffn(q, d, self.wg, self.sg, self.wu, self.su, out_dtype=torch.float32, save=True)
        hq, hd = moe.quantize_act_token(h)
        y, acc2 = moe.int8_matmul(hq, hd, self.wd, self.sd, out_dtype=x.dtype, save=True)
        return y, (q, d, acc, hq, hd, acc2)

    def backward(self, dy, saved):
        q, d, acc, hq, hd, acc2 = saved
        dh_, dsd, _ = moe.int8_matmul_backward(dy, acc2, hd, self.wd, self.sd)
        dx, dsg, dsu = moe.gated_ffn_backward(dh_, acc, d, self.wg, self.sg, self.wu, self.su)
        return dx, dsg, dsu, dsd


@pytest.mark.parametrize("T", [1, 6, 33, 300])
def test_training_step_against_autograd(T):
    """Forward and backward of the whole feed-forward in fp32 against autograd in
    64 bits on the same codes.  Bounds: each of the two products is within 1e-6
    of its magnitude (sum |w v|) by the bounds of dense_helpers (at most 26 u of
    each term, the fixed point 2^-24 of a row's largest for each), and the
    activation's derivative multiplies the first one's error by at most 1.1 |u|."""
    gen = torch.Generator().manual_seed(T)
    H, I = 256, 160
    f = Ffn(gen, H, I)
    x, dy = torch.randn((T, H), generator=gen), torch.randn((T, H), generator=gen)
    y, saved = f.forward(x.cuda())
    grads = f.backward(dy.cuda(), saved)
    q, d, acc, hq, hd, acc2 = (t.cpu().double() for t in saved)
    xs = (q * d[:, None]).requires_grad_()
    sg, su, sd = (s.cpu().double().requires_grad_() for s in (f.sg, f.su, f.sd))
    g, u = xs @ f.qg.double().T * sg, xs @ f.qu.double().T * su
    h = g * torch.sigmoid(g) * u
    hs = (hq * hd[:, None] - h).detach() + h  # the quantised values, the gradient passed through
    y64 = hs @ f.qd.double().T * sd
    want = torch.autograd.grad(y64, (xs, sg, su, sd), dy.double())
    # magnitudes: the same products of magnitudes
    ay = dy.abs().double() * sd.abs()
    ah = ay @ f.qd.double().abs()
    slope = 1.1 * u.abs()
    ax = (ah * slope * sg) @ f.qg.double().abs() + (ah * h.abs().clamp_min(1e-3) / u.abs().clamp_min(1e-3) * su) @ f.qu.double().abs()
    dh.check("y", y, y64.detach(), 8 * dh.U * ((hs.abs() @ f.qd.double().abs().T) * sd + y64.abs()))
    dh.check("dx", grads[0], want[0], 4e-6 * ax.detach() + 1e-12)
    bound = 4e-6 * (ah * slope * (xs.abs() @ f.qg.double().abs().T)).sum(0)
    dh.check("ds_gate", grads[1], want[1], bound.detach())
    bound = 4e-6 * (ah * (g * torch.sigmoid(g)).abs().clamp_min(1e-3) * (xs.abs() @ f.qu.double().abs().T)).sum(0)
    dh.check("ds_up", grads[2], want[2], bound.detach())
    bound = (T + 8) * dh.U * (dy.abs().double() * (hs.abs() @ f.qd.double().abs().T)).sum(0)
    dh.check("ds_down", grads[3], want[3], bound.detach())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """ds of the gated block against central differences of its forward: the
    difference quotient of a smooth function is off by step^2 f'''/6, taken here
    at a thousandth of a scale, and by the forward's own rounding over the step."""
    gen = torch.Generator().manual_seed(5)
    T, K, N = 5, 96, 40
    x, xd, ws, ss, _, dy = dh.inputs(3, T, K, N, 2, torch.float32)
    c = [t.cuda() for t in (x, xd, ws[0], ss[0], ws[1], ss[1], dy)]
    _, acc = moe.gated_ffn(*c[:6], act=act, save=True)
    _, dsg, dsu = moe.gated_ffn_backward(c[6], acc, c[1], c[2], c[3], c[4], c[5], act=act)
    for which, got in ((3, dsg), (5, dsu)):
        step = 1e-3 * c[which]
        quot = []
        for sign in (1, -1):
            a = list(c[:6])
            a[which] = c[which] + sign * step
            quot.append((moe.gated_ffn(*a, act=act) * c[6]).double())
        num = ((quot[0] - quot[1]).sum(0) / (2 * step.double())).cpu()
        mag = ((quot[0].abs() + quot[1].abs()).sum(0) / step.double()).cpu()
        # rounding: 100 u of each value; curvature: (1e-3 |g|)^2, |g| up to a few tens here, of the value's slope
        dh.check("ds", got, num, 100 * dh.U * mag + 1e-2 * num.abs() + 1e-5 * mag)


def test_empty_batches():
    w, s, v0 = (torch.ones((24, 40), dtype=torch.int8, device="cuda"), torch.ones(24, device="cuda"),
                torch.empty(0, device="cuda"))
    x = torch.empty((0, 40), dtype=torch.int8, device="cuda")
    q, d = moe.quantize_act_token(torch.empty((0, 40), device="cuda"))
    assert q.shape == (0, 40) and d.shape == (0,)
    y, acc = moe.int8_matmul(x, v0, w, s, save=True)
    assert y.shape == (0, 24) and acc.shape == (0, 24)
    h, acc2 = moe.gated_ffn(x, v0, w, s, w, s, save=True)
    assert h.shape == (0, 24) and acc2.shape == (2, 0, 24)
    dy = torch.empty((0, 24), device="cuda")
    dx, ds, db = moe.int8_matmul_backward(dy, acc, v0, w, s, bias_grad=True)
    assert dx.shape == (0, 40) and not ds.any() and not db.any()  # sums over no tokens
    dx, dsg, dsu = moe.gated_ffn_backward(dy, acc2, v0, w, s, w, s)
    assert dx.shape == (0, 40) and not dsg.any() and not dsu.any()
    bank = moe.ExpertBank(w.view(torch.uint8)[None], w.view(torch.uint8)[None],
                          torch.ones((1, 40, 24), dtype=torch.uint8, device="cuda"), s[None], s[None],
                          torch.ones((1, 40), device="cuda"))
    assert moe.dense_ffn(torch.empty((0, 40), device="cuda"), bank).shape == (0, 40)


@pytest.mark.parametrize("T", [3, 80, 400])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_of_nothing_and_of_too_much(T, dtype):
    """Zero rows give zero gradients, a row with a NaN or an infinity NaN in its
    own row of dx and in the column sums that it enters, tiny and huge rows theirs."""
    K, N = 144, 96
    x, xd, (w,), (s,), _, dy = dh.inputs(T, T, K, N, 1, DT[dtype])
    dy[0] = 0
    dy[1] = dy[1] * 2.0 ** -100  # the row's fixed point lies below 2^-60
    dy[2] = dy[2] * 2.0 ** 60
    acc = dh.sums64(x, w)
    refs = dh.ref_matmul_backward(dy, acc, xd, w, s, DT[dtype])
    c = [t.cuda() for t in (dy, acc.int(), xd, w, s)]
    got = moe.int8_matmul_backward(*c, bias_grad=True)
    for name, g, (want, tol) in zip(("dx", "ds", "dbias"), got, refs):
        dh.check(name, g, want, tol)
    assert not got[0][0].any()
    bad = c[0].clone()
    bad[0, 5], bad[T - 1, 7] = float("nan"), float("inf")
    dx, ds, db = moe.int8_matmul_backward(bad, *c[1:], bias_grad=True)
    rows = torch.isnan(dx).all(1).cpu()
    assert rows[0] and rows[T - 1] and int(rows.sum()) == 2
    assert torch.equal(dx[1:T - 1], got[0][1:T - 1])
    finite = torch.isfinite(ds) & torch.isfinite(db)
    assert (~finite).nonzero().flatten().tolist() == [5, 7]


def test_gated_backward_of_far_activations():
    """Gates far out (|g| to 1e9): the activation's derivative is 0 or 1 there, never NaN."""
    K, N = 32, 64
    x = torch.full((4, K), 127, dtype=torch.int8)
    x[1], x[3] = -127, 0
    w = torch.full((N, K), 127, dtype=torch.int8)
    xd, s = torch.tensor([1.0, 1.0, 1e3, 1.0]), torch.ones(N)
    dy = torch.ones((4, N))
    c = [t.cuda() for t in (x, xd, w, s, w, s * 1e-6)]
    for act in ("silu", "gelu"):
        h, acc = moe.gated_ffn(*c, act=act, save=True)
        dx, dsg, dsu = moe.gated_ffn_backward(dy.cuda(), acc, c[1], c[2], c[3], c[4], c[5], act=act)
        for t in (h, dx, dsg, dsu):
            assert torch.isfinite(t).all()
        assert not h[1].any() and not dx[1].any()  # g = -5e5: nothing passes


@pytest.mark.parametrize("T", [1, 9, 70, 500])
def test_streams_and_graphs(T):
    """Calls on a side stream, two streams at once, and captured graphs (replayed
    together) give the bits of calls on the current stream."""
    gen = torch.Generator().manual_seed(T)
    f = Ffn(gen, 512, 384)
    bank = moe.ExpertBank(f.wg[None], f.wu[None], f.wd[None], f.sg[None], f.su[None], f.sd[None])
    xs = [torch.randn((T, 512), generator=gen).bfloat16().cuda() for _ in range(2)]
    dys = [torch.randn((T, 512), generator=gen).bfloat16().cuda() for _ in range(2)]

    def step(i):
        y, saved = f.forward(xs[i])
        return (moe.dense_ffn(xs[i], bank), y, *f.backward(dys[i].float(), saved))

    want = [step(0), step(1)]
    again = step(0)
    assert all(torch.equal(a, b) for a, b in zip(want[0], again))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(step(i))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    # the stream argument, with tensors of the current stream
    y = moe.dense_ffn(xs[0], bank, stream=streams[0])
    q, d = moe.quantize_act_token(xs[0], stream=streams[0])
    z = moe.int8_matmul(q, d, f.wg, f.sg, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, want[0][0])
    assert torch.equal(z, moe.int8_matmul(*moe.quantize_act_token(xs[0]), f.wg, f.sg))
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i))
        graphs.append(g)
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
            for t in b:
                t.zero_()
        torch.cuda.synchronize()
    assert moe.dense_device_error() == 0


def test_stream_of_a_chain_of_writes():
    """Each call sees what the one before it wrote, and overwrites what it has read
    (kernels start while their predecessors end)."""
    gen = torch.Generator().manual_seed(1)
    w, s, codes = packed(gen, 512, 512)
    a = torch.randn((64, 512), generator=gen).cuda()
    q = torch.empty((64, 512), dtype=torch.int8, device="cuda")
    want = a
    for _ in range(6):
        qq, dd = moe.quantize_act_token(want)
        torch.cuda.synchronize()
        want = moe.int8_matmul(qq, dd, w, s)
        torch.cuda.synchronize()
    for _ in range(20):
        x = a.clone()
        for _ in range(6):
            qq, dd = moe.quantize_act_token(x)
            q.copy_(qq)
            moe.int8_matmul(q, dd, w, s, out=x)
        assert torch.equal(x, want)


def test_offsets_beyond_32_bits():
    """Results and sums of more than 2^31 elements: the last rows are right."""
    T, K, N = 270_000, 16, 8192
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-127, 128, (T, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    xd, s = torch.rand(T, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    y, acc = moe.int8_matmul(x, xd, w, s, out_dtype=torch.bfloat16, save=True)
    rows = torch.tensor([0, 1, T // 2, 262_143, 262_144, T - 2, T - 1], device="cuda")
    ref = x[rows].double() @ w.double().T
    assert torch.equal(acc[rows].double(), ref)
    ref = ref * xd[rows].double()[:, None] * s.double()
    assert ((y[rows].double() - ref).abs() <= (2 ** -8 + 2 ** -20) * ref.abs()).all()
    dx, ds, _ = moe.int8_matmul_backward(y, acc, xd, w, s)
    ref = (y[rows].double() * s.double()) @ w.double()
    mag = (y[rows].double() * s.double()).abs() @ w.double().abs()
    big = (y[rows].double() * s.double()).abs().amax(1, keepdim=True) * w.double().abs().sum(0)
    assert ((dx[rows].double() - ref).abs() <= 2 ** -8 * ref.abs() + 2 ** -16 * big + 2 ** -20 * mag).all()
    del dx
    some = slice(0, 64)
    ref = (y[:, some].double() * xd.double()[:, None] * acc[:, some].double()).sum(0)
    mag = (y[:, some].double() * xd.double()[:, None] * acc[:, some].double()).abs().sum(0)
    assert ((ds[some].double() - ref).abs() <= 2 ** -14 * mag).all()
    del y, acc, x
    # quantiser: rows past 2^31 elements
    xf = torch.randn((T, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    q, d = moe.quantize_act_token(xf)
    q1, d1 = moe.quantize_act_token(xf[-3:])
    assert torch.equal(q[-3:], q1) and torch.equal(d[-3:], d1)


def test_refusals_of_the_binding():
    x, xd = torch.zeros((4, 32), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    w, s = torch.zeros((8, 32), dtype=torch.int8, device="cuda"), torch.zeros(8, device="cuda")
    acc = torch.zeros((4, 8), dtype=torch.int32, device="cuda")
    dy = torch.zeros((4, 8), device="cuda")
    bad = [
        lambda: moe.int8_matmul(x, xd[:3], w, s),
        lambda: moe.int8_matmul(x, xd, w[:, :31], s),
        lambda: moe.int8_matmul(x, xd, w, s[:7]),
        lambda: moe.int8_matmul(x, xd, w, s.double()),
        lambda: moe.int8_matmul(x, xd, w, s.cpu()),
        lambda: moe.int8_matmul(x, xd, w.cpu(), s),
        lambda: moe.int8_matmul(x.t(), xd, w, s),
        lambda: moe.int8_matmul(x.expand(2, 4, 32), xd, w, s),
        lambda: moe.int8_matmul(x[:1].expand(4, 32), xd, w, s),
        lambda: moe.int8_matmul(x, xd, w, s, bias=s[:4]),
        lambda: moe.int8_matmul(x, xd, w, s, out_dtype=torch.float64),
        lambda: moe.int8_matmul(x, xd, w, s, out=torch.zeros((4, 9), device="cuda")),
        lambda: moe.int8_matmul(x, xd, w, s, out=torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")),
        lambda: moe.gated_ffn(x, xd, w, s, w[:4], s),
        lambda: moe.gated_ffn(x, xd, w, s, w, s, act="relu"),
        lambda: moe.int8_matmul_backward(dy, acc[:3], xd, w, s),
        lambda: moe.int8_matmul_backward(dy, acc.long(), xd, w, s),
        lambda: moe.int8_matmul_backward(dy, acc, None, w, s),
        lambda: moe.int8_matmul_backward(dy.double(), acc, xd, w, s),
        lambda: moe.gated_ffn_backward(dy, acc, xd, w, s, w, s),
        lambda: moe.gated_ffn_backward(dy, acc.expand(2, 4, 8), xd, w, s, w, s),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(moe.MoeError):  # sums past 2^31
        k = torch.zeros((1, 131072), dtype=torch.int8, device="cuda")
        moe.int8_matmul(k, xd[:1], k, s[:1])
