"""Embedding lookup and its gradient against the definitions in 64 bits: small
and large vocabularies, tokens once, often and in every place, both ways of
sorting, layouts, repeated calls.

Bounds: a row's sum of N terms is off by at most N EPS32 of their magnitudes,
the scale's product by one rounding, the addition to a sum by another."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, TINY, U, close, d

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(F32, F32), (F32, BF), (F32, FP), (BF, BF), (FP, FP)]


def rnd(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g).to(dtype)


def text(g, T, n, kind):
    """Tokens: uniform, one in r for the r-th most frequent, all one, sorted or
    falling, or with places that hold none."""
    if kind == "uniform":
        return torch.randint(0, n, (T,), generator=g)
    if kind == "frequent":
        p = 1.0 / torch.arange(2, n + 2, dtype=torch.float64)
        return torch.randperm(n, generator=g)[torch.multinomial(p, T, replacement=True, generator=g)]
    if kind == "one":
        return torch.full((T,), n - 1)
    if kind == "falling":
        return (torch.arange(T).flip(0) * n) // max(T, 1)
    if kind == "runs":            # around the ends of chunks of 8, 16 and 32 places
        out = []
        while len(out) < T:
            r = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 66, 95, 97, 128, 129, 200][int(torch.randint(20, (1,), generator=g))]
            out += [len(out)] * r
        t = torch.unique(torch.tensor(out[:T]), return_inverse=True)[1] % n
        return t[torch.randperm(T, generator=g)]
    if kind == "none":
        return torch.where(torch.arange(T) % 2 == 0, -100, n)
    t = torch.randint(0, n, (T,), generator=g)                # "padded"
    t[torch.rand(T, generator=g) < 0.4] = -1
    t[torch.rand(T, generator=g) < 0.1] = n + 5
    return t


def grad(tokens, dy, n, scale, start=None):
    """(gradient, bound) in 64 bits."""
    m = dy.shape[-1]
    t, v = tokens.reshape(-1).long(), d(dy).reshape(-1, m)
    ok = (t >= 0) & (t < n)
    t, v = t[ok], v[ok]
    w, a = torch.zeros(n, m, dtype=torch.float64), torch.zeros(n, m, dtype=torch.float64)
    w.index_add_(0, t, v)
    a.index_add_(0, t, v.abs())
    cnt = torch.bincount(t, minlength=n).double()[:, None]
    w, off = w * scale, abs(scale) * a * (cnt + 2) * EPS32 + 1e-45
    if start is not None:
        w = w + d(start)
        off = off + w.abs() * EPS32 * (cnt > 0)
    return w, off


@pytest.mark.parametrize("wtype,dtype", PAIRS)
@pytest.mark.parametrize("T,n,m", [(1, 1, 1), (1, 1000, 4096), (5, 3, 7), (33, 100, 8), (70, 515, 100),
                                   (1000, 5000, 515), (3, 40, 20001), (0, 10, 16)])
def test_lookup(T, n, m, wtype, dtype):
    g = torch.Generator().manual_seed(T + n + m)
    w, t = rnd(g, n, m, dtype=wtype), text(g, T, n, "padded")
    for scale in (1.0, 7.3):
        y = d3.embedding(t.cuda(), w.cuda(), scale=scale, dtype=dtype)
        ok = (t >= 0) & (t < n)
        f32 = float(torch.tensor(scale))
        want = torch.where(ok[:, None], d(w)[t.clamp(0, n - 1)] * f32, 0.0)
        # (the product in fp32, then the type)
        off = want.abs() * (U[dtype] + (EPS32 * 1.01 if dtype != F32 else 0)) + TINY[dtype]
        assert y.shape == (T, m) and y.dtype == dtype
        close(y, want, off)
        if scale == 1.0:
            assert torch.equal(y.cpu(), want.to(dtype))
    y = d3.embedding(t.int().cuda(), w.cuda())
    assert y.dtype == wtype and torch.equal(y.cpu(), d(y).to(wtype))


KINDS = ["uniform", "frequent", "one", "falling", "none", "padded", "runs"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,n,m", [(1, 1, 1), (5, 3, 7), (31, 40, 64), (32, 7, 512), (33, 100, 520),
                                   (64, 1, 40), (517, 3000, 515), (1000, 70, 1030), (8192, 500, 40),
                                   (8193, 70, 36), (20000, 300, 20), (70000, 40000, 8),
                                   (9000, 70001, 8), (40, 5000, 1), (3, 9999, 2), (50, 3000, 3),
                                   (700, 4000, 130), (100, 300, 4100), (65, 50, 40), (128, 50, 40),
                                   (6000, 3000, 2600), (30000, 3000, 1100), (64, 30, 520), (90, 20, 513), (300, 50, 1027),
                                   (40, 9, 258), (33, 10, 5), (70, 6, 65026)])
def test_gradient(T, n, m, kind):
    g = torch.Generator().manual_seed(T + n + m)
    dtype = (BF, FP, F32)[(T + m) % 3]
    t, dy = text(g, T, n, kind), rnd(g, T, m, dtype=dtype)
    t = t.int() if T % 2 else t
    scale = 1.0 if n % 2 else 0.3
    f32 = float(torch.tensor(scale))
    want, off = grad(t, dy, n, f32)
    got = d3.embedding_grad(t.cuda(), dy.cuda(), n, scale=scale)
    assert got.dtype == F32 and got.shape == (n, m)
    close(got, want, off)
    again = d3.embedding_grad(t.cuda(), dy.cuda(), n, scale=scale)
    assert torch.equal(got, again)
    # summed into a buffer: rows without tokens keep their bits, here NaN
    ok = torch.zeros(n, dtype=torch.bool)
    ok[t[(t >= 0) & (t < n)].long()] = True
    start = rnd(g, n, m)
    start[~ok] = float("nan")
    out = start.cuda()
    assert d3.embedding_grad(t.cuda(), dy.cuda(), n, scale=scale, out=out, accumulate=True) is out
    assert torch.isnan(out.cpu()[~ok]).all()
    want, off = grad(t, dy, n, f32, start)
    close(out[ok.cuda()], want[ok], off[ok] + EPS32 * want[ok].abs())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T", [100, 9001])
def test_layouts(T, accumulate):
    g = torch.Generator().manual_seed(T)
    n, m = 300, 77
    t, dy, w = text(g, T, n, "frequent").cuda(), rnd(g, T, m, dtype=BF).cuda(), rnd(g, n, m).cuda()
    want = d3.embedding_grad(t, dy, n, out=w.clone(), accumulate=accumulate)
    look = d3.embedding(t, w, dtype=BF)
    for ld, off in ((m + 3, 1), (m, 1), (80, 8)):
        buf = torch.full((T * ld + off + 9,), float("nan"), dtype=BF, device="cuda")
        v = buf.as_strided((T, m), (ld, 1), off)
        v.copy_(dy)
        wb = torch.full((n * ld + off + 9,), 7.0, device="cuda")
        wv = wb.as_strided((n, m), (ld, 1), off)
        wv.copy_(w)
        assert torch.equal(d3.embedding(t, wv, dtype=BF), look)
        d3.embedding_grad(t, v, n, out=wv, accumulate=accumulate)
        assert torch.equal(wv, want)
        mask = torch.ones_like(wb, dtype=torch.bool)
        mask.as_strided(wv.shape, wv.stride(), off).fill_(False)
        assert (wb[mask] == 7).all()


def test_no_tokens():
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    dy = torch.empty(0, 24, dtype=BF, device="cuda")
    assert not d3.embedding_grad(e, dy, 100).any()
    out = torch.ones(100, 24, device="cuda")
    d3.embedding_grad(e, dy, 100, out=out, accumulate=True)
    assert (out == 1).all()


def test_offsets_past_32_bits():
    """A table past 2^32 bytes and 2^31 elements, and its gradient."""
    n, m = 1 << 20, 2056
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free GPU memory")
    w = torch.zeros(n, m, device="cuda")
    w[n - 1], w[n // 2] = 3.0, 2.0
    t = torch.tensor([n - 1, 0, n // 2, n - 1], device="cuda")
    y = d3.embedding(t, w, dtype=BF)
    assert [float(r[0]) for r in y] == [3, 0, 2, 3] and (y == y[:, :1]).all()
    d3.embedding_grad(t, y, n, out=w)
    assert float(w[n - 1, m - 1]) == 6 and float(w[n // 2, 0]) == 2
    assert int((w != 0).any(1).sum()) == 2


@pytest.mark.parametrize("wtype", [F32, BF])
def test_differentiable_form(wtype):
    g = torch.Generator().manual_seed(1)
    w = rnd(g, 50, 24, dtype=wtype).cuda().requires_grad_(True)
    t, dy = text(g, 18, 50, "padded").view(3, 6).cuda(), rnd(g, 3, 6, 24, dtype=BF).cuda()
    y = d3.embedding_layer(t, w, scale=1.5, dtype=BF)
    assert y.shape == (3, 6, 24) and torch.equal(y, d3.embedding(t, w.detach(), 1.5, BF))
    y.backward(dy)
    assert w.grad.dtype == wtype
    assert torch.equal(w.grad, d3.embedding_grad(t, dy, 50, 1.5).to(wtype))
    w.grad = None
    d3.embedding_layer(t, w, dtype=BF).sum().backward()       # an expanded gradient
    want, _ = grad(t.cpu(), torch.ones(3, 6, 24), 50, 1.0)
    assert torch.equal(w.grad.cpu().double(), want)
    # each entry's derivative is the scale times its tokens: by differences of the sum
    e = torch.zeros(50, 24, dtype=wtype, device="cuda")
    e[int(t[t >= 0][0].clamp_max(49)), 3] = 1.0
    a = d3.embedding(t, w.detach() * 0 + e, 1.0, wtype).double().sum()
    assert float(a) == float((e.double() * want.cuda()).sum())


def test_captured():
    g = torch.Generator().manual_seed(2)
    for T in (300, 9000):
        t, dy = text(g, T, 200, "frequent").cuda(), rnd(g, T, 40, dtype=BF).cuda()
        out = torch.empty(200, 40, device="cuda")
        d3.embedding_grad(t, dy, 200, out=out)
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            d3.embedding_grad(t, dy, 200, out=out)
            y = d3.embedding(t, out, dtype=BF)
        for _ in range(4):
            t.copy_(text(g, T, 200, "padded"))
            dy.copy_(rnd(g, T, 40))
            graph.replay()
            torch.cuda.synchronize()
            want = d3.embedding_grad(t, dy, 200)
            assert torch.equal(out, want) and torch.equal(y, d3.embedding(t, want, dtype=BF))


def test_refusals():
    w, t = torch.zeros(9, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = torch.zeros(4, 8, dtype=BF, device="cuda")
    for error, f in (
            (TypeError, lambda: d3.embedding(t, w.double())),
            (TypeError, lambda: d3.embedding(t, w.cpu())),
            (TypeError, lambda: d3.embedding(t, w.to(BF), dtype=FP)),
            (TypeError, lambda: d3.embedding(t, w, dtype=torch.float64)),
            (TypeError, lambda: d3.embedding(t.float(), w)),
            (TypeError, lambda: d3.embedding(t.cpu(), w)),
            (ValueError, lambda: d3.embedding(t, w.t())),
            (ValueError, lambda: d3.embedding(t, w[0])),
            (d3.Dion3Error, lambda: d3.embedding(t, w, scale=float("nan"))),
            (TypeError, lambda: d3.embedding_grad(t, dy.double(), 9)),
            (TypeError, lambda: d3.embedding_grad(t.float(), dy, 9)),
            (ValueError, lambda: d3.embedding_grad(t[:3], dy, 9)),
            (ValueError, lambda: d3.embedding_grad(t, dy, 9, accumulate=True)),
            (ValueError, lambda: d3.embedding_grad(t, dy, 8, out=w)),
            (TypeError, lambda: d3.embedding_grad(t, dy, 9, out=w.to(BF))),
            (d3.Dion3Error, lambda: d3.embedding_grad(t, dy, 0)),
            (d3.Dion3Error, lambda: d3.embedding_grad(t, dy, 9, scale=float("inf")))):
        with pytest.raises(error):
            f()
