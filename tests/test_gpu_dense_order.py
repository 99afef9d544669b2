"""The dense int8 operators where calls meet: operands rewritten in place between
calls (kernels start while their predecessors end), several threads, and rows at
addresses off the 16-byte grid in batches of any size.  All results are compared
bit for bit with calls that have the device to themselves."""
import threading

import pytest
import torch

from quantized_routed_expert_group_b200 import moe

pytestmark = pytest.mark.gpu


def make(gen, T, K, N, n=1):
    def i8(*shape):
        return torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
    xs = [i8(T, K) for _ in range(n)]
    dys = [torch.randn((T, N), generator=gen, device="cuda").bfloat16() for _ in range(n)]
    ws = [i8(N, K) for _ in range(2)]
    ss = [torch.rand(N, generator=gen, device="cuda") * 1e-3 for _ in range(2)]
    return xs, dys, torch.rand(T, generator=gen, device="cuda") * 0.02, ws, ss


def step(x, dy, xd, ws, ss):
    y, a1 = moe.int8_matmul(x, xd, ws[0], ss[0], save=True)
    h, a2 = moe.gated_ffn(x, xd, ws[0], ss[0], ws[1], ss[1], save=True)
    return (y, h, *moe.int8_matmul_backward(dy, a1, xd, ws[0], ss[0], bias_grad=True),
            *moe.gated_ffn_backward(dy, a2, xd, ws[0], ss[0], ws[1], ss[1]))


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T,K,N", [(9, 256, 512), (100, 128, 1040), (700, 512, 2048), (2500, 64, 333)])
@pytest.mark.parametrize("graph", [False, True])
def test_operands_rewritten_in_place(T, K, N, graph):
    """Column sums start beside the product and read what the row kernel has just written; each round
    rewrites the same memory."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    n = 8
    xs, dys, xd, ws, ss = make(gen, T, K, N, n)
    want = []
    for x, dy in zip(xs, dys):
        torch.cuda.synchronize()
        want.append(step(x, dy, xd, ws, ss))
        torch.cuda.synchronize()
    x, dy = torch.empty_like(xs[0]), torch.empty_like(dys[0])

    def chain():
        got = []
        for i in range(n):
            x.copy_(xs[i])
            dy.copy_(dys[i])
            got.append(step(x, dy, xd, ws, ss))
        return got

    if not graph:
        for _ in range(5):
            got = chain()
            assert all(same(a, b) for a, b in zip(got, want))
        return
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for _ in range(5):
        for r in got:
            for t in r:
                t.zero_()
        g.replay()
        assert all(same(a, b) for a, b in zip(got, want))
    assert moe.dense_device_error() == 0


@pytest.mark.parametrize("T", [1, 7, 16])
def test_weights_rewritten_before_a_feed_forward(T):
    """The second kernel of a few tokens' feed-forward reads its weights before the first ends."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    H, I, n = 1024, 512, 6
    u8 = [[torch.randint(0, 256, s, generator=gen, device="cuda", dtype=torch.uint8)
           for s in ((1, I, H), (1, I, H), (1, H, I))] for _ in range(n)]
    scales = [torch.rand((1, r), generator=gen, device="cuda") * 1e-3 for r in (I, I, H)]
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    want = []
    for w in u8:
        torch.cuda.synchronize()
        want.append(moe.dense_ffn(x, moe.ExpertBank(*w, *scales)))
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    bank = moe.ExpertBank(*(torch.empty_like(w) for w in u8[0]), *scales)
    for _ in range(20):
        got = []
        for w in u8:
            for dst, src in zip((bank.w_gate, bank.w_up, bank.w_down), w):
                dst.copy_(src)
            got.append(moe.dense_ffn(x, bank))
        assert same(got, want)


def test_threads():
    """Calls from several threads at once, each on its own stream."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    jobs = [make(gen, T, K, N) for T, K, N in ((5, 512, 256), (33, 100, 300), (300, 1000, 500), (1200, 512, 1024))]
    want = [step(xs[0], dys[0], xd, ws, ss) for xs, dys, xd, ws, ss in jobs]
    torch.cuda.synchronize()
    failures = []

    def work(job, ref):
        try:
            xs, dys, xd, ws, ss = job
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    if not same(step(xs[0], dys[0], xd, ws, ss), ref):
                        failures.append("other bits")
        except Exception as e:  # (an assertion in a thread is lost)
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures
    assert moe.dense_device_error() == 0


# rows of a multiple of 16 codes at addresses and strides that are none, from small batches to such as would
# be copied if their length were odd
@pytest.mark.parametrize("T,K,N", [(40, 512, 300), (300, 1024, 1040), (2000, 1024, 1501)])
@pytest.mark.parametrize("offset,pitch", [(8, 0), (4, 4), (0, 8), (1, 0), (0, 2)])
def test_views_off_the_grid(T, K, N, offset, pitch):
    gen = torch.Generator(device="cuda").manual_seed(T)
    xs, dys, xd, ws, ss = make(gen, T, K, N)
    want = step(xs[0], dys[0], xd, ws, ss)

    def view(t):
        rows, cols = t.shape
        ld = cols + 16 + pitch
        buf = torch.zeros(rows * ld + offset, dtype=t.dtype, device="cuda")
        v = buf[offset:].view(rows, ld)[:, :cols]
        v.copy_(t)
        return v

    assert same(step(view(xs[0]), dys[0], xd, [view(w) for w in ws], ss), want)
    assert moe.dense_device_error() == 0
