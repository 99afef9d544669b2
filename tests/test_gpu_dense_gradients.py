"""Gradients of the dense int8 operators on rows of a wide range: one element far
above the others (a softmax less its target over a vocabulary, outliers), a loud
channel of the gated block.

Bounds (u = 2^-24; v: the gradient rows, dy s, of which dx = v w):
  each v is off by its own few roundings (3u of |v|, or what dense_helpers
  derives for the gated block's), by the multiplier's, the scale's and two
  products' (4u), and by half a unit of the row's fixed point, m / (2 D), m the
  row's largest magnitude.  The digits of an integer r in a balanced base 256
  add up to at most 3 |r| in magnitude, so the planes' sums, each converted to
  fp32 and joined by fused multiply-adds and one product, round by at most
  (P + 1) 3u <= 15u of sum |v w|.  Together 24u sum |v w|, and the fixed point.
  That one's errors are sums of N roundings of at most c = m |w| / (2 D): by
  Hoeffding's inequality they pass 7 sqrt(sum c^2) with a probability of 2
  exp(-49/2) < 5e-11 a result.  D is 8355600 for 16-bit gradients (24 bits) and
  2139060224 for fp32 (32 bits): for a softmax, whose other elements sum to the
  largest, that is at most 2^-12 (16 bits) and 16u (fp32) of sum |v w|.
Results are rounded once: half a step of their type.
"""
import pytest
import torch

import dense_helpers as dh
from quantized_routed_expert_group_b200 import moe

pytestmark = pytest.mark.gpu

DT = dh.DTYPES
D = {"fp32": 2139060224.0, "bf16": 8355600.0, "fp16": 8355600.0}


def codes(gen, rows, cols):
    """int8 codes with a mean of a third of their spread."""
    return (torch.randn((rows, cols), generator=gen, device="cuda") * 36 + 12).round().clamp(-127, 127).to(torch.int8)


def wide_rows(gen, T, N, kind):
    if kind == "softmax":  # times a loss scale
        p = torch.softmax(0.3 * torch.randn((T, N), generator=gen, device="cuda"), 1)
        target = torch.randint(0, N, (T,), generator=gen, device="cuda")
        p[torch.arange(T, device="cuda"), target] -= 1
        return 512 * p
    v = torch.randn((T, N), generator=gen, device="cuda") * torch.exp(torch.randn((T, 1), generator=gen, device="cuda"))
    v[torch.arange(T), torch.randint(0, N, (T,), generator=gen, device="cuda")] *= kind
    return v


def check_dx(name, got, vs, evs, ws, dtype):
    dx, tol, squares = 0, 0, 0
    for v, ev, w in zip(vs, evs, ws):
        w = w.double()
        dx = dx + v @ w
        tol = tol + (ev + 24 * dh.U * v.abs()) @ w.abs()
        squares = squares + (w * w).sum(0)
    m = torch.stack([v.abs().amax(1) for v in vs]).amax(0)[:, None]
    tol = tol + 7 * m / (2 * D[dtype]) * squares.sqrt() + dh.rounding(DT[dtype], dx)
    over = dx.abs() > torch.finfo(DT[dtype]).max + tol  # past fp16's last number: an infinity
    assert torch.equal(got[over].double(), dx[over].sign() * float("inf"))
    dh.check(name, got.masked_fill(over, 0), dx.masked_fill(over, 0).cpu(), tol.cpu())


# single CTAs and pairs, rows of codes on the 16-byte grid and off it
@pytest.mark.parametrize("T,K,N", [(20, 64, 128256), (200, 128, 128256), (17, 101, 32000), (300, 64, 32000),
                                   (9, 48, 131071), (70, 72, 8192)])
@pytest.mark.parametrize("dtype", list(DT))
def test_matmul_backward_of_a_softmax(T, K, N, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    w, s = codes(gen, N, K), (torch.rand(N, generator=gen, device="cuda") + 0.5) / 64
    dy = wide_rows(gen, T, N, "softmax").to(DT[dtype])
    v = dy.double() * s.double()
    dx = moe.int8_matmul_backward(dy, None, None, w, s)[0]
    check_dx("dx", dx, [v], [3 * dh.U * v.abs()], [w], dtype)
    assert moe.dense_device_error() == 0


@pytest.mark.parametrize("T,K,N", [(40, 256, 6144), (300, 64, 6144)])
@pytest.mark.parametrize("loud", [1, 30, 300, 10000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dx_is_as_exact_as_a_plain_product(T, K, N, loud, dtype):
    """The error of dx over a batch against that of the fp32 product, rounded once.  Both round
    nearly the same numbers, so the second is the rounding's; what the first adds is the fixed
    point's, independent of it: m sqrt(N) / (2 sqrt(3) D) of rms(w), against |dx| of about
    |v| rms(w) >= m rms(w): at most 3e-6 of |dx|, where the rounding leaves 2e-4 or more."""
    gen = torch.Generator(device="cuda").manual_seed(T + loud)
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    s = (torch.rand(N, generator=gen, device="cuda") + 0.5) / 1e4
    top = torch.finfo(DT[dtype]).max / 2
    dy = wide_rows(gen, T, N, loud).clamp(-top, top).to(DT[dtype])  # (fp16 ends at 65,504)
    want = (dy.double() * s.double()) @ w.double()
    plain = ((dy.float() * s) @ w.float()).to(DT[dtype])
    dx = moe.int8_matmul_backward(dy, None, None, w, s)[0]
    error = [float((t.double() - want).norm() / want.norm()) for t in (dx, plain)]
    assert error[0] <= 1.02 * error[1], error


@pytest.mark.parametrize("T,K,N", [(20, 64, 32000), (300, 96, 8192), (17, 101, 5001), (40, 64, 65535), (400, 128, 2048)])
@pytest.mark.parametrize("act,dtype", [("silu", "bf16"), ("gelu", "fp16"), ("silu", "fp32")])
def test_gated_backward_of_a_softmax_with_a_loud_channel(T, K, N, act, dtype):
    """Both matrices share a row's fixed point; a loud channel of one of them leaves the rest intact."""
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    ws = [codes(gen, N, K) for _ in range(2)]
    ss = [(torch.rand(N, generator=gen, device="cuda") + 0.5) / (50 * K ** 0.5) for _ in range(2)]
    ss[1][N // 3] *= 1000
    x = torch.randint(-127, 128, (T, K), generator=gen, device="cuda", dtype=torch.int8)
    xd = torch.rand(T, generator=gen, device="cuda") * 0.02 + 1e-3
    acc = torch.stack([x.double() @ w.double().T for w in ws])
    dy = wide_rows(gen, T, N, "softmax").to(DT[dtype])
    got = moe.gated_ffn_backward(dy, acc.int(), xd, ws[0], ss[0], ws[1], ss[1], act=act)
    xs = [xd.double()[:, None] * a for a in acc]
    g, u = (t * s.double() for t, s in zip(xs, ss))
    z, a, da, da_mag, da_tiny = dh.act64(act, g)
    rel, d = (30 + 16 * z.abs()) * dh.U, dy.double()
    dg, du = d * u * da, d * a
    eg = (d * u).abs() * (da_mag * rel + da_tiny * dh.TINY)
    eu = du.abs() * rel + d.abs() * (g.abs() + 1) * dh.TINY
    check_dx("dx", got[0], [dg * ss[0].double(), du * ss[1].double()], [eg * ss[0].double(), eu * ss[1].double()], ws,
             dtype)
    assert moe.dense_device_error() == 0


# columns that leave one CTA the whole batch: many of them, and an odd number
@pytest.mark.parametrize("T,N", [(20000, 9600), (60000, 2401), (70000, 33), (3000, 640)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_matmul_column_sums_of_a_long_batch(T, N, dtype):
    """ds and dbias over batches of one sign, each column's terms alike, so that a long fp32 sum
    would round the same way at every step.  Bounds: a term rounds three times, 32 of them are
    summed in fp32, what follows is in fp64 but for one rounding a chunk and one of the result:
    (3 + 31 + 2) u of the terms' sum."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    K = 16
    dy = (torch.rand(N, generator=gen, device="cuda") + 0.1).to(DT[dtype]).expand(T, N).contiguous()
    acc = torch.randint(1, 200_000, (N,), generator=gen, device="cuda", dtype=torch.int32).expand(T, N).contiguous()
    xd = torch.full((T,), 0.0123, device="cuda")
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    s = torch.rand(N, generator=gen, device="cuda")
    _, ds, db = moe.int8_matmul_backward(dy, acc, xd, w, s, bias_grad=True)
    want = T * dy[0].double() * xd[0].double() * acc[0].double()
    dh.check("ds", ds, want.cpu(), 36 * dh.U * want.cpu())
    want = T * dy[0].double()
    dh.check("dbias", db, want.cpu(), 36 * dh.U * want.cpu())


# a group of columns a thread, four of them, rows of any length, single columns
@pytest.mark.parametrize("T,N", [(300000, 64), (60000, 6400), (60000, 4099), (200000, 333), (9473, 2048), (5, 512)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gated_column_sums_of_a_long_batch(T, N, dtype):
    """The same for the scales of the gated block.  Bounds: the term's own error (dense_helpers), 31
    additions in fp32, and what follows in fp64 but for one rounding a partial sum and one of the
    result, 2u; 3u for the term's last products."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    K = 16
    dy = (torch.rand(N, generator=gen, device="cuda") + 0.1).to(DT[dtype]).expand(T, N).contiguous()
    acc = torch.randint(20_000, 200_000, (2, 1, N), generator=gen, device="cuda", dtype=torch.int32)
    xd = torch.full((T,), 0.0123, device="cuda")
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    ss = [torch.full((N,), v, device="cuda") for v in (4e-4, 3e-4)]  # g up to 1, u up to 0.7
    _, *got = moe.gated_ffn_backward(dy, acc.expand(2, T, N).contiguous(), xd, w, ss[0], w, ss[1])
    d, x = dy[0].double(), xd[0].double() * acc[:, 0].double()
    g, u = x[0] * ss[0].double(), x[1] * ss[1].double()
    z, a, da, da_mag, _ = dh.act64("silu", g)
    rel = (30 + 16 * z.abs()) * dh.U
    for name, t, want, e in (("ds_gate", got[0], d * u * da * x[0], d * u * da_mag * rel * x[0]),
                             ("ds_up", got[1], d * a * x[1], d * a * rel * x[1])):
        dh.check(name, t, T * want.cpu(), T * (e + 36 * dh.U * want).cpu())


class Linear(torch.autograd.Function):
    """The product with its backward pass, as a program joins them."""

    @staticmethod
    def forward(ctx, x, w, s, bias):
        q, d = moe.quantize_act_token(x)
        y, acc = moe.int8_matmul(q, d, w, s, bias=bias, out_dtype=x.dtype, save=True)
        ctx.save_for_backward(acc, d, w, s)
        return y

    @staticmethod
    def backward(ctx, dy):
        dx, ds, dbias = moe.int8_matmul_backward(dy, *ctx.saved_tensors, bias_grad=True)
        return dx, None, ds, dbias


def test_an_autograd_function_of_the_calls():
    """Leaves are refused outside, taken inside, and get the backward pass's gradients."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, K, N = 40, 96, 50
    x = torch.randn((T, K), generator=gen, device="cuda").requires_grad_()
    s = torch.rand(N, generator=gen, device="cuda").requires_grad_()
    bias = torch.randn(N, generator=gen, device="cuda").requires_grad_()
    w, dy = codes(gen, N, K), torch.randn((T, N), generator=gen, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        moe.quantize_act_token(x)
    y = Linear.apply(x, w, s, bias)
    y.backward(dy)
    with torch.no_grad():
        q, d = moe.quantize_act_token(x)
        want, acc = moe.int8_matmul(q, d, w, s, bias=bias, save=True)
        grads = moe.int8_matmul_backward(dy, acc, d, w, s, bias_grad=True)
    assert torch.equal(y, want)
    for leaf, g in zip((x, s, bias), grads):
        assert torch.equal(leaf.grad, g)
