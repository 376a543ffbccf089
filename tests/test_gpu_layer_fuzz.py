"""Random sizes, strides, alignments and types of the layer operators, with
operands surrounded by NaN: products of small whole numbers exactly, row
operators against themselves on contiguous copies and the 64-bit formulas."""
import random

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, U

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def size(r, hi):
    """1 .. hi, spread over the logarithm; multiples of 8 and 128, and any."""
    v = max(1, int(round(hi ** r.random())))
    k = r.random()
    return max(1, v // 128 * 128) if k < 0.25 else max(1, v // 8 * 8) if k < 0.5 else v


def place(r, t):
    """t's values at a random row stride and element offset, NaN around them."""
    T, m = t.shape
    ld, off = r.choice([(m, 0), (m, 1), (m + 1, 0), (m + 8 - m % 8, 8), (m + r.randint(1, 40), r.randint(0, 9))])
    buf = torch.full((max(1, T) * ld + off + 16,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf.as_strided((T, m), (ld, 1), off)
    v.copy_(t)
    return v


def ints(g, *shape, dtype):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("seed", range(40))
def test_random_products(seed):
    r = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for _ in range(4):
        t = r.choice([BF, FP])
        T, n, m = size(r, 3000), size(r, 3000), size(r, 3000)
        x, w, dz = ints(g, T, m, dtype=t), ints(g, n, m, dtype=t), ints(g, T, n, dtype=t)
        X, W, Z = place(r, x), place(r, w), place(r, dz)
        what = (seed, T, n, m, t)
        b = ints(g, n, dtype=r.choice([t, torch.float32])) if r.random() < 0.5 else None
        res = ints(g, T, n, dtype=t) if r.random() < 0.5 else None
        act = r.choice(["none", "relu"])
        y, z = d3.linear(X, W, bias=b, act=act, residual=None if res is None else place(r, res),
                         return_preact=True)
        want = x.double() @ w.double().t().contiguous()
        want = want if b is None else want + b.double()
        assert torch.equal(z, want.to(t)), what
        want = want.clamp_min(0) if act == "relu" else want
        want = want if res is None else want + res.double()
        assert torch.equal(y, want.to(t)), what
        assert torch.equal(d3.linear_grad_input(Z, W), (dz.double() @ w.double()).to(t)), what
        want = dz.double().t().contiguous() @ x.double()
        assert torch.equal(d3.linear_grad_weight(Z, X).double(), want), what
        out = place(r, torch.ones(n, m, device="cuda"))
        d3.linear_grad_weight(Z, d3.pack_f8(X), out=out, accumulate=True)
        assert torch.equal(out.double(), want + 1), what


@pytest.mark.parametrize("seed", range(40))
def test_random_rows(seed):
    r = random.Random(1000 + seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for _ in range(4):
        t = r.choice([BF, FP])
        T, m = size(r, 4000), size(r, 20000)
        x, res, dy, dh = (torch.randn(T, m, generator=g, device="cuda").to(t) for _ in range(4))
        w = (1 + 0.1 * torch.randn(m, generator=g, device="cuda")).to(r.choice([t, torch.float32]))
        what = (seed, T, m, t)
        a = d3.add_rms_norm(x, w, residual=res, pack=True)
        b = d3.add_rms_norm(place(r, x), w, residual=place(r, res), pack=True)
        for u, v in zip((*a[:3], a[3].q.view(torch.uint8), a[3].scale),
                        (*b[:3], b[3].q.view(torch.uint8), b[3].scale)):
            assert torch.equal(u, v), what
        p = d3.pack_f8(a[0])
        assert torch.equal(p.q.view(torch.uint8), a[3].q.view(torch.uint8)), what
        h = a[1].double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * w.double()
        assert ((a[0].double() - y).abs() <= y.abs() * (U[t] + 128 * EPS32) + 2.0 ** -24).all(), what
        ga = d3.add_rms_norm_grad(dy, a[1], a[2], w, dh=dh)
        gb = d3.add_rms_norm_grad(place(r, dy), place(r, a[1]), a[2], w, dh=place(r, dh))
        assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1]), what
        u = h * a[2].double()[:, None]
        want = (dy.double() * u).sum(0)
        lim = (dy.double() * u).abs().sum(0) * (T + 4) * EPS32 + 1e-30
        assert ((ga[1].double() - want).abs() <= lim).all(), what
        act = r.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        da = d3.act_grad(dy, x, act, bias=True)
        db = d3.act_grad(place(r, dy), place(r, x), act, bias=True)
        assert torch.equal(da[0], db[0]) and torch.equal(da[1], db[1]), what
