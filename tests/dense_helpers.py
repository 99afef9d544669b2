"""The dense int8 operators in 64 bits, with the error that their documented
arithmetic may have, and seeded inputs.

Bounds (u = 2^-24, half a step of fp32; e(t) = eps/2 of the result's type):
  product: the integer sum's conversion, the product of the scales and the
    product of both round once each, the bias' sum once: 4u (|acc xd s| + |y|).
  activation: g carries 3u; z(g) a few roundings more (gelu: at most 6 of its
    own and 3 times g's for the cube), all of them relative, so exp(-|z|) is off
    by at most 16 |z| u relative; expf, the division and the products add less
    than 24 u.  |delta act| <= |act| (24 + 16 |z|) u, and the same for each
    addend of its derivative.
  gradient rows: an element v is off by its own arithmetic, delta_v, and by the
    fixed point: at most m / (2 D) (m: the row's largest; D: 32639 or 8355600),
    and 2u of v from the scaling.  dx then has sum |w| of these, and 8u sum |w v|
    from the join of the digits and the scales.
  column sums: each term's own error, and one rounding for each of the rows that
    one partial sum holds (ceil(T / 592) at 148 SMs; T is taken, which is larger).
Results are rounded once to their type: e(t) |y|, and half the smallest number.
"""
import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -147  # see "activation"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
G0, G1 = 2 * math.sqrt(2 / math.pi), 0.044715


def rounding(dtype, y):
    """Half a step of the type at y, and half its smallest positive number."""
    info = torch.finfo(dtype)
    return info.eps / 2 * y.abs() + info.smallest_normal * info.eps / 2


def codes(gen, rows, cols):
    """Random int8 codes with saturated ones among them (-128 too: the packers never write it, the products take it)."""
    q = torch.randint(-127, 128, (rows, cols), generator=gen, dtype=torch.int16)
    q[0, : max(1, cols // 3)] = 127
    q[-1, cols // 2:] = -128
    return q.to(torch.int8)


def inputs(seed, T, K, N, mats, dtype):
    gen = torch.Generator().manual_seed(seed)
    x = codes(gen, T, K)
    xd = torch.rand(T, generator=gen) * 0.02 + 1e-3
    ws = [codes(gen, N, K) for _ in range(mats)]
    # scales that bring g and u to a few units: |acc| is about 74^2 sqrt(K)
    ss = [(torch.rand(N, generator=gen) + 0.5) / (50.0 * math.sqrt(K)) for _ in range(mats)]
    bias = torch.randn(N, generator=gen)
    dy = (torch.randn((T, N), generator=gen) * torch.exp(torch.randn((T, 1), generator=gen))).to(dtype)
    return x, xd, ws, ss, bias, dy


def sums64(x, w):
    return x.double() @ w.double().T  # exact: every partial sum is an integer below 2^53


def ref_matmul(x, xd, w, s, bias, dtype):
    acc = sums64(x, w)
    prod = acc * xd.double()[:, None] * s.double()
    y = prod if bias is None else prod + bias.double()
    return acc, y, 4 * U * (prod.abs() + y.abs()) + rounding(dtype, y)


def act64(act, g):
    z = g if act == "silu" else G0 * (g + G1 * g ** 3)
    dz = torch.ones_like(g) if act == "silu" else G0 * (1 + 3 * G1 * g ** 2)
    sig = torch.sigmoid(z)
    dsig = sig * torch.sigmoid(-z)
    return z, g * sig, sig + g * dsig * dz, sig + (g * dsig * dz).abs(), 1 + (g * dz).abs()


def ref_gated(x, xd, ws, ss, act, dtype):
    ag, au = sums64(x, ws[0]), sums64(x, ws[1])
    g, u = ag * xd.double()[:, None] * ss[0].double(), au * xd.double()[:, None] * ss[1].double()
    z, a = act64(act, g)[:2]
    h = a * u
    return torch.stack([ag, au]), h, \
        (30 + 16 * z.abs()) * U * h.abs() + u.abs() * (g.abs() + 1) * TINY + rounding(dtype, h)


def _dx(vs, evs, ws, dtype):
    D = 8355600.0 if dtype == torch.float32 else 32639.0
    m = torch.stack([v.abs().amax(1) for v in vs]).amax(0)[:, None]
    dx = sum(v @ w.double() for v, w in zip(vs, ws))
    tol = sum((ev + 10 * U * v.abs() + 0.51 * m / D) @ w.double().abs() for v, ev, w in zip(vs, evs, ws))
    return dx, tol + rounding(dtype, dx)


def ref_matmul_backward(dy, acc, xd, w, s, dtype):
    dy = dy.double()
    v = dy * s.double()
    dx, tx = _dx([v], [2 * U * v.abs()], [w], dtype)
    T = dy.shape[0]
    term = dy * xd.double()[:, None] * acc
    return (dx, tx), (term.sum(0), (T + 8) * U * term.abs().sum(0) + 1e-45), \
        (dy.sum(0), (T + 8) * U * dy.abs().sum(0) + 1e-45)


def ref_gated_backward(dh, acc, xd, ws, ss, act, dtype):
    dh, T = dh.double(), dh.shape[0]
    xg, xu = xd.double()[:, None] * acc[0], xd.double()[:, None] * acc[1]
    g, u = xg * ss[0].double(), xu * ss[1].double()
    z, a, da, da_mag, da_tiny = act64(act, g)
    rel = (30 + 16 * z.abs()) * U
    dg, du = dh * u * da, dh * a
    edg = (dh * u).abs() * (da_mag * rel + da_tiny * TINY)
    edu = du.abs() * rel + dh.abs() * (g.abs() + 1) * TINY
    dx, tx = _dx([dg * ss[0].double(), du * ss[1].double()], [edg * ss[0].double(), edu * ss[1].double()], ws, dtype)
    out = [(dx, tx)]
    for d, e, x in ((dg, edg, xg), (du, edu, xu)):
        out.append(((d * x).sum(0), (e * x.abs()).sum(0) + (T + 8) * U * (d * x).abs().sum(0) + 1e-45))
    return out


def check(name, got, want, tol):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off; worst "
                           f"{float(((got - want).abs() / tol).max()):.3g} of the bound at "
                           f"{tuple(int(i) for i in bad.nonzero()[0])}")
