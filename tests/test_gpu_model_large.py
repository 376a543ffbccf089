"""Calls whose reads or writes pass the 256 MB cache, against the same calls on
parts that do not: bit for bit where a row stands for itself."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests import test_gpu_embedding as emb
from tests.layer_ref import EPS32, close

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("not enough free GPU memory")
    yield
    torch.cuda.empty_cache()


def rnd(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D,r,gap", [(BF, 128, 128, 0), (FP, 96, 32, 8), (BF, 80, 20, 0), (FP, 100, 36, 3)])
def test_heads(dtype, D, r, gap, interleaved):
    g = torch.Generator(device="cuda").manual_seed(D + r)
    hq, hk = 48, 5
    h = hq + hk
    T = int(70e6) // (2 * h * D) + 1
    x, dy = rnd(g, T, h, D + gap, dtype=dtype)[..., :D], rnd(g, T, h, D + gap, dtype=dtype)[..., :D]
    assert 2 * T * h * D > 64e6
    w, v = rnd(g, D), rnd(g, D)
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda")
    fr = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).cuda()

    def both(a, b):
        q, k = x[a:b, :hq], x[a:b, hq:]
        y = d3.qk_norm_rope(q, k, w, v, pos[a:b], fr, interleaved=interleaved)
        return y + d3.qk_norm_rope_grad(dy[a:b, :hq], dy[a:b, hq:], q, k, w, v, pos[a:b], fr,
                                        interleaved=interleaved)

    whole = both(0, T)
    dw = [torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2)]
    for a in range(0, T, 1000):
        b = min(T, a + 1000)
        part = both(a, b)
        for i in range(4):
            assert torch.equal(whole[i][a:b], part[i]), (i, a)
        for i in range(2):
            dw[i] += part[4 + i].double()
    # The terms are the same numbers in both; a term goes through at most 100
    # additions (of a lane at most 40: the tokens' batches over 3000 waves; of
    # the lanes 6, the waves 3, the workgroups 18), and is du hat with du at
    # most sqrt(2) times the head's largest |dy|.
    xd, top = x.double(), dy.double().abs().amax(-1, keepdim=True)
    terms = 2 ** 0.5 * top * xd.abs() / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-6)
    for i, part in enumerate((terms[:, :hq], terms[:, hq:])):
        assert ((whole[4 + i].double() - dw[i]).abs() <= 2 * 100 * EPS32 * part.sum((0, 1))).all()


def test_embedding():
    g = torch.Generator(device="cuda").manual_seed(1)
    for dtype, m in ((BF, 4096), (F32, 2050), (FP, 4099)):
        w = rnd(g, 5000, m, dtype=dtype)
        T = int(96e6) // (m * w.element_size()) + 77
        t = torch.randint(-1, 5001, (T,), generator=g, device="cuda")
        ok = (t >= 0) & (t < 5000)
        want = w[t.clamp(0, 4999)] * ok[:, None]
        assert torch.equal(d3.embedding(t, w), want), dtype


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_clip_into_sums(dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    shapes = [(5001, 4099), (3, 7), (2500, 8000), (33,)]
    grads, sums = [rnd(g, *s, dtype=dtype) for s in shapes], [rnd(g, *s) for s in shapes]
    n = sum(v.numel() for v in grads)
    while n * (4 + grads[0].element_size()) <= 288e6:
        grads.append(rnd(g, 4000, 4001, dtype=dtype))
        sums.append(rnd(g, 4000, 4001))
        n += grads[-1].numel()
    before = [m.clone() for m in sums]
    norm = d3.clip_grad_norm(grads, 100.0, into=sums)
    exact = sum(float(v.double().square().sum()) for v in grads) ** 0.5
    assert abs(float(norm) - exact) <= exact * EPS32 * 1.001
    c = 100.0 / exact
    for v, b, m in zip(grads, before, sums):
        want = b.double() + c * v.double()
        assert ((m.double() - want).abs() <= want.abs() * EPS32 * 1.0001 + 1e-45).all()


def test_rows_far_apart():
    """The last token's row of each sequence, and tables with such rows."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n, S = 32001, 70
    far = rnd(g, 5, S, n, dtype=BF)
    assert S * n > 1 << 21
    x = far[:, -1]
    near = x.contiguous()
    t = torch.randint(0, n, (5,), generator=g, device="cuda")
    a, b = (d3.log_probs(v, t, entropy=True, top=7) for v in (x, near))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ones, keep = torch.ones(5, device="cuda"), far[:, :-1].clone()
    want = d3.log_probs_grad(ones, near, t, b[1], entropy=b[2], dentropy=ones)
    d3.log_probs_grad(ones, x, t, a[1], entropy=a[2], dentropy=ones, out=x)
    assert torch.equal(x, want) and torch.equal(far[:, :-1], keep)
    w = rnd(g, 6, S, n)[:, 3]
    tokens = torch.tensor([5, 0, 5, 7, 1], device="cuda")
    y = d3.embedding(tokens, w)
    assert torch.equal(y, d3.embedding(tokens, w.contiguous()))
    dy = rnd(g, 5, S, n, dtype=BF)[:, 0]
    grad = d3.embedding_grad(tokens, dy.contiguous(), 6)
    assert torch.equal(d3.embedding_grad(tokens, dy, 6, out=w), grad)


@pytest.mark.parametrize("kind", ["uniform", "frequent", "padded", "runs"])
@pytest.mark.parametrize("T,n,m", [(262144, 300, 4), (262145, 300, 4), (300001, 70001, 9)])
def test_embedding_gradient_of_many_tokens(T, n, m, kind):
    """Around the number of tokens from which the digits' scan is a launch."""
    g = torch.Generator().manual_seed(T + n)
    t, dy = emb.text(g, T, n, kind), emb.rnd(g, T, m, dtype=BF)
    want, off = emb.grad(t, dy, n, 1.0)
    got = d3.embedding_grad(t.cuda(), dy.cuda(), n)
    close(got, want, off, kind)
    assert torch.equal(d3.embedding_grad(t.int().cuda(), dy.cuda(), n), got)


def test_two_streams_and_threads():
    """Calls at once, from two threads on two streams, each with its own results."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(4)
    n, T, D = 20001, 600, 128
    fr = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()

    def inputs():
        return dict(x=rnd(g, T, n, dtype=BF), t=torch.randint(-1, n, (T,), generator=g, device="cuda"),
                    q=rnd(g, T, 12, D, dtype=BF), k=rnd(g, T, 2, D, dtype=BF), w=rnd(g, D),
                    p=torch.randint(0, 9999, (T,), generator=g, device="cuda"), e=rnd(g, T, 300, dtype=BF),
                    grads=[rnd(g, 500, 300, dtype=BF) for _ in range(70)])

    def run(a):
        lp = d3.log_probs(a["x"], a["t"], entropy=True, top=64)
        dx = d3.log_probs_grad(lp[0], a["x"], a["t"], lp[1], entropy=lp[2], dentropy=lp[2])
        y = d3.qk_norm_rope(a["q"], a["k"], a["w"], a["w"], a["p"], fr)
        dy = d3.qk_norm_rope_grad(*y, a["q"], a["k"], a["w"], a["w"], a["p"], fr)
        de = d3.embedding_grad(a["t"], a["e"], n)
        sums = [torch.zeros(500, 300, device="cuda") for _ in a["grads"]]
        norm = d3.clip_grad_norm(a["grads"], 1.0, into=sums)
        return [*lp, dx, *y, *dy, de, norm, *sums]

    both = [inputs(), inputs()]
    want = [run(a) for a in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    got, bad = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                got[i] = [run(both[i]) for _ in range(8)]
        except Exception as e:              # (a thread's own failure would not be the test's)
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not bad
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(u, v) for u, v in zip(outs, want[i])), i
