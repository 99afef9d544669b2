"""Cases and plain forms of the dense int8 operators: the matrix product with
scales for each token and channel, the gated feed-forward block, their backward
passes, and the feed-forward that runs them together.

Weights are rows of int8 codes with an fp32 scale each (as pack_weights gives
them, in uint8 storage); activations are rows of int8 codes with an fp32 scale
each.  Gradients reach the dequantised activations, the row scales and the
bias; the codes are constants.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}

# The layer's shape in this repository: hidden 6144, intermediate 2048.


def listed():
    return [
        # one decoded token through a projection: latency and the weights' stream
        {"name": "matmul_decode", "op": "matmul", "T": 1, "K": 6144, "N": 2048, "dtype": "bf16", "bias": False},
        # a small serving batch through the down projection, fp32 results
        {"name": "matmul_batch16", "op": "matmul", "T": 16, "K": 2048, "N": 6144, "dtype": "fp32", "bias": False},
        # odd sizes: rows that are no multiple of 16 bytes, a ragged batch, a bias
        {"name": "matmul_ragged", "op": "matmul", "T": 333, "K": 1000, "N": 777, "dtype": "fp16", "bias": True},
        # a long prompt through a square projection
        {"name": "matmul_prefill", "op": "matmul", "T": 4096, "K": 6144, "N": 6144, "dtype": "bf16", "bias": False},
        # the gated block for one decoded token
        {"name": "gated_decode", "op": "gated", "T": 1, "K": 6144, "N": 2048, "dtype": "bf16", "act": "silu"},
        # the gated block for a long prompt
        {"name": "gated_prefill", "op": "gated", "T": 4096, "K": 6144, "N": 2048, "dtype": "bf16", "act": "silu"},
        # a training step of the gated block: forward with what the backward needs, then the backward
        {"name": "gated_train", "op": "gated_train", "T": 2048, "K": 6144, "N": 2048, "dtype": "bf16", "act": "silu"},
        # the same at odd sizes, gradients in fp32
        {"name": "gated_train_ragged", "op": "gated_train", "T": 300, "K": 1000, "N": 500, "dtype": "fp32",
         "act": "gelu"},
        # a training step of the down projection with a bias
        {"name": "matmul_train", "op": "matmul_train", "T": 2048, "K": 2048, "N": 6144, "dtype": "bf16", "bias": True},
        # a short fp32 training batch with an odd number of channels
        {"name": "matmul_train_short", "op": "matmul_train", "T": 77, "K": 512, "N": 1023, "dtype": "fp32",
         "bias": True},
        # the whole feed-forward for the four tokens of a speculative verify
        {"name": "ffn_verify", "op": "ffn", "T": 4, "K": 6144, "N": 2048, "dtype": "bf16", "act": "silu"},
        # the whole feed-forward for a prompt of a thousand tokens
        {"name": "ffn_prefill", "op": "ffn", "T": 1024, "K": 6144, "N": 2048, "dtype": "bf16", "act": "silu"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "gated", "gated", "gated_train", "matmul_train", "ffn"])
    case = {"op": op, "T": _spread(rng, 1, 4096), "K": _spread(rng, 64, 8192), "N": _spread(rng, 32, 6144),
            "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    if rng.random() < 0.6:  # most models' rows are multiples of 32
        case["K"] = -(-case["K"] // 32) * 32
        case["N"] = -(-case["N"] // 32) * 32
    most = 4096 * 6144 * 6144
    while case["T"] * case["K"] * case["N"] * (4 if op == "gated_train" else 3 if op == "ffn" else 2) > most:
        case["T"] = max(1, case["T"] // 2)
    if op == "ffn":  # the packed bank's rows are multiples of 32, and its result is a 16-bit type in serving
        case["K"] = -(-case["K"] // 32) * 32
        case["N"] = -(-case["N"] // 32) * 32
        case["dtype"] = rng.choice(["bf16", "fp16"])
    if op.startswith("matmul"):
        case["bias"] = rng.random() < 0.5
    else:
        case["act"] = rng.choice(["silu", "gelu"])
    return case


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _quantise_rows(x):
    """Per-row symmetric int8 in fp32 steps: d = amax/127, q = round-half-away(x * (1/d))."""
    x = x.float()
    amax = x.abs().amax(dim=-1, keepdim=True)
    live = amax >= 2.0 ** -112
    d = torch.where(live, amax / torch.full_like(amax, 127.0), torch.zeros_like(amax))
    v = x * torch.where(live, torch.reciprocal(d), torch.zeros_like(d))
    low = v.abs().floor()
    low = low + (v.abs() - low >= 0.5).float()
    q = torch.where(v < 0, -low, low).clamp(-127, 127)
    return q, d.squeeze(-1)


def _weights(gen, rows, cols):
    w = torch.randn((rows, cols), generator=gen, device="cuda") * 0.02
    q, s = _quantise_rows(w)
    return q.to(torch.int8).view(torch.uint8), s


def _activations(gen, rows, cols):
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.01  # a hundredth of the channels are loud
    return torch.where(loud, x * 8.0, x)


def _gradient(gen, rows, cols, dtype):
    """Rows of different sizes; the padded tail of a batch has none."""
    size = 1e-3 * torch.exp(torch.randn((rows, 1), generator=gen, device="cuda"))
    dy = torch.randn((rows, cols), generator=gen, device="cuda") * size
    dy[rows - rows // 16:] = 0
    return dy.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    T, K, N, dtype = case["T"], case["K"], case["N"], DTYPES[case["dtype"]]
    st = {"op": case["op"], "dtype": dtype, "act": case.get("act")}
    x = _activations(gen, T, K)
    if case["op"] == "ffn":
        st["x"] = x.to(dtype)
        st["wg"], st["sg"] = _weights(gen, N, K)
        st["wu"], st["su"] = _weights(gen, N, K)
        st["wd"], st["sd"] = _weights(gen, K, N)
        return st
    q, st["xd"] = _quantise_rows(x)
    st["xq"] = q.to(torch.int8)
    if case["op"].startswith("matmul"):
        st["w"], st["s"] = _weights(gen, N, K)
        st["bias"] = torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
    else:
        st["wg"], st["sg"] = _weights(gen, N, K)
        st["wu"], st["su"] = _weights(gen, N, K)
    if case["op"].endswith("train"):
        st["dy"] = _gradient(gen, T, N, dtype)
    return st


# ----------------------------------------------------------------------------
# Plain forms, in fp32
# ----------------------------------------------------------------------------
def _codes(w):
    return w.view(torch.int8).float()


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


_G0, _G1 = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def _act(act, g):
    return g * _sigmoid(g if act == "silu" else _G0 * (g + _G1 * g * g * g))


def _act_grad(act, g):
    sig = _sigmoid(g if act == "silu" else _G0 * (g + _G1 * g * g * g))
    slope = 1.0 if act == "silu" else _G0 * (1.0 + 3.0 * _G1 * g * g)
    return sig + g * sig * (1.0 - sig) * slope


def _plain_matmul(xq, xd, w, s, bias):
    acc = xq.float() @ _codes(w).T
    y = acc * (xd[:, None] * s)
    return acc, y if bias is None else y + bias


def _plain_gated(xq, xd, wg, sg, wu, su, act):
    acc_g, acc_u = xq.float() @ _codes(wg).T, xq.float() @ _codes(wu).T
    g, u = acc_g * (xd[:, None] * sg), acc_u * (xd[:, None] * su)
    return acc_g, acc_u, g, u, _act(act, g) * u


def _run_plain(st):
    op, dtype = st["op"], st["dtype"]
    if op == "ffn":
        q, d = _quantise_rows(st["x"])
        h = _plain_gated(q, d, st["wg"], st["sg"], st["wu"], st["su"], st["act"])[4]
        q, d = _quantise_rows(h)
        return {"y": _plain_matmul(q, d, st["wd"], st["sd"], None)[1].to(dtype)}
    if op.startswith("matmul"):
        acc, y = _plain_matmul(st["xq"], st["xd"], st["w"], st["s"], st["bias"])
        out = {"y": y.to(dtype)}
        if op.endswith("train"):
            dy = st["dy"].float()
            out["dx"] = ((dy * st["s"]) @ _codes(st["w"])).to(dtype)
            out["ds"] = (dy * acc * st["xd"][:, None]).sum(0)
            if st["bias"] is not None:
                out["dbias"] = dy.sum(0)
        return out
    acc_g, acc_u, g, u, h = _plain_gated(st["xq"], st["xd"], st["wg"], st["sg"], st["wu"], st["su"], st["act"])
    out = {"h": h.to(dtype)}
    if op.endswith("train"):
        dh = st["dy"].float()
        dg, du = dh * u * _act_grad(st["act"], g), dh * _act(st["act"], g)
        out["dx"] = ((dg * st["sg"]) @ _codes(st["wg"]) + (du * st["su"]) @ _codes(st["wu"])).to(dtype)
        out["ds_gate"] = (dg * acc_g * st["xd"][:, None]).sum(0)
        out["ds_up"] = (du * acc_u * st["xd"][:, None]).sum(0)
    return out


# ----------------------------------------------------------------------------
# The framework's calls
# ----------------------------------------------------------------------------
def _run_own(st):
    from quantized_routed_expert_group_b200 import moe
    op, dtype = st["op"], st["dtype"]
    if op == "ffn":
        bank = moe.ExpertBank(st["wg"][None], st["wu"][None], st["wd"][None], st["sg"][None], st["su"][None],
                              st["sd"][None])
        return {"y": moe.dense_ffn(st["x"], bank, act=st["act"])}
    if op == "matmul":
        return {"y": moe.int8_matmul(st["xq"], st["xd"], st["w"], st["s"], bias=st["bias"], out_dtype=dtype)}
    if op == "matmul_train":
        y, acc = moe.int8_matmul(st["xq"], st["xd"], st["w"], st["s"], bias=st["bias"], out_dtype=dtype, save=True)
        dx, ds, dbias = moe.int8_matmul_backward(st["dy"], acc, st["xd"], st["w"], st["s"],
                                                 bias_grad=st["bias"] is not None)
        out = {"y": y, "dx": dx, "ds": ds}
        if dbias is not None:
            out["dbias"] = dbias
        return out
    if op == "gated":
        return {"h": moe.gated_ffn(st["xq"], st["xd"], st["wg"], st["sg"], st["wu"], st["su"], act=st["act"],
                                   out_dtype=dtype)}
    h, acc = moe.gated_ffn(st["xq"], st["xd"], st["wg"], st["sg"], st["wu"], st["su"], act=st["act"],
                           out_dtype=dtype, save=True)
    dx, dsg, dsu = moe.gated_ffn_backward(st["dy"], acc, st["xd"], st["wg"], st["sg"], st["wu"], st["su"],
                                          act=st["act"])
    return {"h": h, "dx": dx, "ds_gate": dsg, "ds_up": dsu}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


def work(case):
    T, K, N, e = case["T"], case["K"], case["N"], DTYPES[case["dtype"]].itemsize
    op = case["op"]
    if op == "ffn":
        return {"bytes": 2 * T * K * e + 3 * N * K + 8 * N + 4 * K, "flops": 6 * T * K * N}
    m = 1 if op.startswith("matmul") else 2  # weight matrices
    size = T * K + 4 * T + m * (N * K + 4 * N) + T * N * e + (4 * N if case.get("bias") else 0)
    flops = 2 * m * T * K * N
    if op.endswith("train"):
        size += T * N * e + T * K * e + 4 * m * N + (4 * N if case.get("bias") else 0)
        flops *= 2
    return {"bytes": size, "flops": flops}


# ----------------------------------------------------------------------------
# The definition in 64 bits; gradients by differentiating it
# ----------------------------------------------------------------------------
def _exact_quantise(x64):
    """Codes and scales by the definition, whose scale, reciprocal and product are fp32 numbers."""
    amax = x64.abs().max(dim=1).values
    d = (amax / 127.0).float()
    d = torch.where(amax < 2.0 ** -112, torch.zeros_like(d), d)
    inv = torch.where(d > 0, (1.0 / d.double()).float(), torch.zeros_like(d))
    v = (x64 * inv.double()[:, None]).float().double()
    q = torch.sign(v) * torch.floor(v.abs() + 0.5)
    return q.clamp(-127.0, 127.0), d.double()


def _exact_act(act, g):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def _w64(w):
    return w.view(torch.int8).double()


def exact(case, seed):
    st = prepare(case, seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "ffn":
        q, d = _exact_quantise(st["x"].double())
        x = q * d[:, None]
        g = torch.einsum("tk,nk->tn", x, _w64(st["wg"])) * st["sg"].double()
        u = torch.einsum("tk,nk->tn", x, _w64(st["wu"])) * st["su"].double()
        # the hidden values are fp32 numbers before they are quantised
        q, d = _exact_quantise((_exact_act(case["act"], g) * u).float().double())
        return {"y": torch.einsum("tn,kn->tk", q * d[:, None], _w64(st["wd"])) * st["sd"].double()}
    train = op.endswith("train")
    x = (st["xq"].double() * st["xd"].double()[:, None]).requires_grad_(train)
    if op.startswith("matmul"):
        scales = [st["s"].double().requires_grad_(train)]
        b = None if st["bias"] is None else st["bias"].double().requires_grad_(train)
        y = torch.einsum("tk,nk->tn", x, _w64(st["w"])) * scales[0]
        y = y if b is None else y + b
        names, leaves = ["dx", "ds"] + (["dbias"] if b is not None else []), [x] + scales + ([b] if b is not None else [])
        out = {"y": y.detach()}
    else:
        scales = [st["sg"].double().requires_grad_(train), st["su"].double().requires_grad_(train)]
        g = torch.einsum("tk,nk->tn", x, _w64(st["wg"])) * scales[0]
        u = torch.einsum("tk,nk->tn", x, _w64(st["wu"])) * scales[1]
        y = _exact_act(case["act"], g) * u
        names, leaves = ["dx", "ds_gate", "ds_up"], [x] + scales
        out = {"h": y.detach()}
    if train:
        out.update(zip(names, torch.autograd.grad(y, leaves, st["dy"].double())))
    return out
