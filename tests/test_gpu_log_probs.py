"""Log probabilities, entropy, best alternatives and their gradient against the
formulas in 64 bits: vocabularies around the pieces a row is cut into, masked
and degenerate rows, ties, layouts.

Bounds, in units of EPS32: exp(d) is off by 3 |d| + 2 of itself (d, its product
with log2 e and the constant rounded once each, the exponential), twice that
over the pieces' own maxima; a sum goes through at most 64 additions; a
logarithm and each further operation is rounded once."""
import math

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, TINY, U, close, d

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = [BF, FP, F32]
SIZES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 100), (70, 515), (4, 1000), (3, 2047), (3, 8192), (2, 8193),
         (9, 32000), (2, 50257), (3, 131072), (2, 131073), (1, 400001), (1, 1 << 20), (0, 100),
         (3000, 40), (1024, 8200),
         (1500, 20001)]


def logits(g, T, n, dtype, std=3.0):
    x = torch.randn(T, n, generator=g) * std
    if T and n > 20:
        x.scatter_add_(1, torch.randint(0, n, (T, 5), generator=g), torch.full((T, 5), 9.0))
    return x.to(dtype)


class Want:
    """The formulas in 64 bits, and bounds."""

    def __init__(self, x, targets, scale):
        z = d(x) * scale
        self.n = x.shape[1]
        self.m = z.amax(1, keepdim=True)
        dz = z - self.m
        self.l = torch.logsumexp(dz, 1, keepdim=True)
        self.q = dz - self.l
        self.p = torch.exp(self.q)
        pd = torch.where(self.p > 0, self.p * dz, torch.zeros_like(dz))
        pdd = torch.where(self.p > 0, self.p * dz * dz, torch.zeros_like(dz))
        self.H = (self.l - pd.sum(1, keepdim=True))[:, 0]
        ed, edd = -pd.sum(1), pdd.sum(1)
        self.lse = (self.m + self.l)[:, 0]
        # of the sum of exponentials, relative; of l
        self.s_off = (6 * ed + 70) * EPS32
        self.l_off = self.s_off + 3 * self.l[:, 0].abs() * EPS32 + 2 * EPS32
        self.H_off = self.l_off + (6 * edd + 74 * ed + 2 * self.H.abs()) * EPS32 + ed * self.s_off
        j = targets.long()
        self.ok = (j >= 0) & (j < self.n)
        dt = dz.gather(1, j.clamp(0, self.n - 1)[:, None])[:, 0]
        self.logp = torch.where(self.ok, dt - self.l[:, 0], 0.0)
        self.logp_off = self.l_off + (dt.abs() + self.logp.abs()) * EPS32
        self.dz, self.j = dz, j

    def grad(self, g, gh, scale):
        """The gradient and the bound of its error before rounding."""
        hot = torch.zeros_like(self.p)
        hot[self.ok, self.j[self.ok]] = 1.0
        g = torch.where(self.ok, d(g), 0.0)[:, None]
        w = g * (hot - self.p)
        size = g.abs() * self.p
        if gh is not None:
            gh = d(gh)[:, None]
            lnp = torch.where(self.p > 0, self.q, 0.0)
            w = w - gh * self.p * (lnp + self.H[:, None])
            size = size + gh.abs() * self.p * (lnp.abs() + self.H[:, None].abs())
        off = (4 * (self.q.abs() + self.dz.abs()).clamp_max(300) + 24) * EPS32 + self.l_off[:, None]
        more = 0.0 if gh is None else gh.abs() * self.p * (self.H_off[:, None] + off)
        return scale * w, scale * (size * off + more + g.abs() * hot * 4 * EPS32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", SIZES)
def test_log_probs_and_gradient(T, n, dtype):
    g = torch.Generator().manual_seed(T + n)
    x = logits(g, T, n, dtype)
    targets = torch.randint(0, n, (T,), generator=g)
    if T > 2:
        targets[1], targets[2] = -100, n                # places without a token
    scale = 0.75 if n % 2 else 1.0
    t = targets.int() if n % 3 else targets
    w = Want(x, targets, scale)
    logp, stats, H, none, none2 = d3.log_probs(x.cuda(), t.cuda(), scale=scale, entropy=True)
    assert none is None and none2 is None and stats.shape == (T, 2) and logp.dtype == F32
    close(d(stats).sum(1), w.lse, w.l_off + 2 * w.lse.abs() * 2.0 ** -53, "lse")
    close(stats[:, 0], w.m[:, 0], w.m[:, 0].abs() * EPS32, "m")
    # (the sums are relative to the rounded maximum, so l moves against it)
    close(logp, w.logp, w.logp_off, "logp")
    close(H, w.H, w.H_off, "entropy")
    a = d3.log_probs(x.cuda(), scale=scale)
    assert a[0] is None and a[2] is None and torch.equal(a[1], stats)
    gl, gh = torch.randn(T, generator=g), torch.randn(T, generator=g)
    for with_h in (False, True):
        dx = d3.log_probs_grad(gl.cuda(), x.cuda(), t.cuda(), stats, scale=scale, entropy=H,
                               dentropy=gh.cuda() if with_h else None)
        want, off = w.grad(gl, gh if with_h else None, scale)
        assert dx.dtype == dtype
        close(dx, want, (want.abs() + off) * U[dtype] + off + TINY[dtype] + 1e-37, ("dx", with_h))
    want, off = w.grad(torch.zeros(T), gh, scale)
    dx = d3.log_probs_grad(None, x.cuda(), None, stats, scale=scale, entropy=H, dentropy=gh.cuda())
    close(dx, want, (want.abs() + off) * U[dtype] + off + TINY[dtype] + 1e-37, "entropy's alone")


def best(x, top):
    """Stable order: NaN first, then by value, equal ones by index."""
    v = x.double().nan_to_num(nan=math.inf, posinf=1e300)          # NaN above infinity
    return torch.sort(v, dim=1, descending=True, stable=True)[1][:, :top]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [s for s in SIZES if s[0]])
def test_best_alternatives(T, n, dtype):
    g = torch.Generator().manual_seed(3 * T + n)
    x = logits(g, T, n, dtype)
    x[0, : n // 2] = x[0, 0]                            # long ties
    targets = torch.randint(0, n, (T,), generator=g)
    w = Want(x, targets, 1.25)
    for top in sorted({1, min(5, n), min(20, n), min(64, n)}):
        logp, stats, H, tl, ti = d3.log_probs(x.cuda(), targets.cuda(), scale=1.25, entropy=True, top=top)
        at = best(x, top)
        assert ti.dtype == torch.int64 and torch.equal(ti.cpu(), at), top
        want = w.q.gather(1, at)
        close(tl, want, w.l_off[:, None] + (w.dz.gather(1, at).abs() + want.abs()) * EPS32, "top")
        close(logp, w.logp, w.logp_off, "logp")
        close(H, w.H, w.H_off, "entropy")
        plain = d3.log_probs(x.cuda(), targets.cuda(), scale=1.25, entropy=True)
        for a, b in zip(plain[:3], (logp, stats, H)):   # (the pieces' order of joining differs)
            assert torch.allclose(a, b, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [50, 2048, 9000, 140000])
def test_best_of_hard_rows(n, dtype):
    """Rows that leave too many candidates: constant, few values, in order, one
    lane's columns, minus infinity all but a few, zeros of both signs, NaN."""
    g = torch.Generator().manual_seed(n)
    i = torch.arange(n, dtype=torch.float32)
    rows = [torch.full((n,), 2.5), torch.randint(-2, 3, (n,), generator=g).float(), i / n * 8, -i / n * 8,
            torch.where(i % 512 < 8, 5.0, 0.0) + torch.rand(n, generator=g),
            torch.where(i % 16 == 3, i.frac() + 1.0, torch.tensor(-math.inf)),
            torch.where(i < 3, -i, torch.tensor(-math.inf)), torch.where(i % 2 == 0, 0.0, -0.0),
            torch.full((n,), -math.inf), -torch.rand(n, generator=g),
            torch.full((n,), torch.finfo(dtype).min)]
    x = torch.stack(rows).to(dtype)
    nan = x[1].clone()
    nan[n // 3], nan[n - 1] = math.nan, -math.nan
    inf = x[1].clone()
    inf[5], inf[n - 2] = math.inf, math.inf
    many = torch.full((n,), math.nan).to(dtype)
    x = torch.cat([x, nan[None], inf[None], many[None]])
    for top in (1, 17, 50):
        _, stats, _, tl, ti = d3.log_probs(x.cuda(), top=top)
        assert torch.equal(ti.cpu(), best(x, top)), top
        assert torch.isnan(tl[-3:]).all() and not torch.isnan(tl[:-3]).any()
        assert (tl[8] == -math.inf).all() and (tl[6, 3:] == -math.inf).all()
        assert abs(float(tl[0, 0]) + math.log(n)) <= 1e-5 * math.log(n) + 1e-6


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [3, 100, 9000])
def test_masked_rows(n, dtype):
    """All minus infinity: no probability, no gradient.  The type's lowest
    value everywhere: 1 / n each.  Both among ordinary values: nothing."""
    low = torch.finfo(dtype).min
    x = torch.zeros(5, n, dtype=dtype)
    x[0] = -math.inf
    x[1] = low
    x[2, 1:] = low
    x[3, 1:] = -math.inf
    x[4, : n - 1] = low
    x[4, n - 1] = -math.inf
    t = torch.tensor([0, 1, 0, 2, 0])
    ones = torch.ones(5).cuda()
    logp, stats, H, tl, ti = d3.log_probs(x.cuda(), t.cuda(), entropy=True, top=2)
    assert logp[0] == -math.inf and stats[0].tolist() == [-math.inf, 0.0] and H[0] == 0
    u = math.log(n)
    assert abs(float(logp[1]) + u) <= 1e-6 * (1 + u) and abs(float(H[1]) - u) <= 1e-6 * (1 + u)
    if dtype != FP:
        assert float(logp[2]) == 0 and float(H[2]) == 0 and float(tl[2, 1]) <= -1e38
    else:
        assert float(logp[2]) == 0 and float(H[2]) == 0 and float(tl[2, 1]) == low
    assert float(logp[3]) == -math.inf and float(H[3]) == 0 and float(tl[3, 0]) == 0
    v = math.log(n - 1)
    assert abs(float(logp[4]) + v) <= 1e-6 * (1 + v) and abs(float(H[4]) - v) <= 1e-6 * (1 + v)
    dx = d3.log_probs_grad(ones, x.cuda(), t.cuda(), stats, entropy=H, dentropy=ones)
    assert torch.isfinite(dx).all() and not dx[0].any()
    p = torch.full((n,), 1 / n, dtype=torch.float64)
    want = -p
    want[1] += 1                                        # uniform: no gradient of the entropy
    close(dx[1], want, want.abs() * (U[dtype] + 100 * EPS32) + 3 * (1 + u) * EPS32 / n * 40)
    assert not dx[2].any()
    assert float(dx[3, 0]) == -1 and float(dx[3, 2]) == 1 and float(dx[3].double().sum()) == 0
    assert float(dx[4, n - 1]) == 0


def test_rows_with_nan_and_infinity():
    x = torch.zeros(4, 9000)
    x[1, 8999], x[2, 0], x[3, 5] = math.nan, math.inf, 3e38
    t = torch.zeros(4, dtype=torch.int64)
    for scale in (1.0, 2.0):                            # 3e38 * 2 is infinite
        logp, stats, H, _, _ = d3.log_probs(x.cuda(), t.cuda(), scale=scale, entropy=True)
        dx = d3.log_probs_grad(torch.ones(4).cuda(), x.cuda(), t.cuda(), stats, scale=scale)
        for bad in (1, 2) if scale == 1 else (1, 2, 3):
            assert math.isnan(logp[bad]) and math.isnan(H[bad]) and torch.isnan(dx[bad]).all()
        assert math.isfinite(logp[0]) and torch.isfinite(dx[0]).all()
    # a place without a token asks nothing of its row
    t[1] = -100
    dx = d3.log_probs_grad(torch.ones(4).cuda(), x.cuda(), t.cuda(), stats)
    assert float(logp[1]) != 0 and not dx[1].any()
    assert float(d3.log_probs(x.cuda(), t.cuda())[0][1]) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [5, 333, 20001])
def test_layouts_and_in_place(n, dtype):
    g = torch.Generator().manual_seed(n)
    x = logits(g, 6, n, dtype)
    t = torch.randint(0, n, (6,), generator=g).cuda()
    gl, gh = torch.randn(6, generator=g).cuda(), torch.randn(6, generator=g).cuda()
    a = d3.log_probs(x.cuda(), t, entropy=True, top=4)
    ga = d3.log_probs_grad(gl, x.cuda(), t, a[1], entropy=a[2], dentropy=gh)
    for ld, off in ((n + 3, 1), (n, 1), (n + 8, 8)):
        buf = torch.full((6 * ld + off + 9,), float("nan"), dtype=dtype, device="cuda")
        v = buf.as_strided((2, 3, n), (3 * ld, ld, 1), off)
        v.copy_(x.view(2, 3, n))
        b = d3.log_probs(v, t.view(2, 3), entropy=True, top=4)
        for p, q in zip(a, b):
            assert torch.equal(p, q.reshape(p.shape))
        s = v[0]                                        # over the logits themselves
        out = d3.log_probs_grad(gl[:3], s, t[:3], a[1][:3], entropy=a[2][:3], dentropy=gh[:3], out=s)
        assert out is s and torch.equal(s, ga[:3])
        assert torch.equal(v[1].cpu(), x[3:])
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask.as_strided(v.shape, v.stride(), off).fill_(False)
        assert torch.isnan(buf[mask]).all()


def test_offsets_past_32_bits():
    """Rows past 2^31 logits."""
    T, n = 70000, 32768
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough free GPU memory")
    x = torch.zeros(T, n, dtype=BF, device="cuda")
    x[-1, 77] = 12.0
    t = torch.full((T,), 77, device="cuda")
    logp, stats, _, tl, ti = d3.log_probs(x, t, top=2)
    want = 12 - math.log(math.exp(12.0) + n - 1)
    assert abs(float(logp[-1]) - want) <= 1e-5 and abs(float(logp[0]) + math.log(n)) <= 1e-5
    assert ti[-1].tolist() == [77, 0] and ti[-2].tolist() == [0, 1]
    d3.log_probs_grad(torch.ones(T, device="cuda"), x, t, stats, out=x)
    assert abs(float(x[-1, 77]) - (1 - math.exp(want))) <= 2.0 ** -8 and float(x[-2, 77]) > 0.99


def test_gradient_by_differences():
    g = torch.Generator().manual_seed(9)
    x = logits(g, 2, 40, F32)
    t, gl, gh = torch.tensor([3, 30]), torch.randn(2, generator=g), torch.randn(2, generator=g)
    y = x.cuda().requires_grad_(True)
    logp, H = d3.token_log_probs(y, t.cuda(), scale=0.8, entropy=True)
    (logp @ gl.cuda() + H @ gh.cuda()).backward()

    def f(v):
        lp = torch.log_softmax(v * 0.8, 1)
        return (lp.gather(1, t[:, None])[:, 0] * d(gl)).sum() - ((lp.exp() * lp).sum(1) * d(gh)).sum()

    e = 1e-5
    for i in range(2):
        for j in range(0, 40, 3):
            s = torch.zeros(2, 40, dtype=torch.float64)
            s[i, j] = e
            num = float(f(d(x) + s) - f(d(x) - s)) / (2 * e)
            assert abs(float(y.grad[i, j]) - num) <= 1e-5


def test_differentiable_form():
    g = torch.Generator().manual_seed(10)
    x, t = logits(g, 12, 500, BF).view(3, 4, 500).cuda(), torch.randint(0, 500, (3, 4), generator=g).cuda()
    t[0, 0] = -100
    logp, stats, H, _, _ = d3.log_probs(x, t, entropy=True)
    y = x.clone().requires_grad_(True)
    a, none = d3.token_log_probs(y, t)
    assert none is None and torch.equal(a, logp)
    (-a.sum() / 11).backward()                          # an expanded gradient
    want = d3.log_probs_grad(torch.full((3, 4), -1 / 11).cuda(), x, t, stats)
    assert torch.equal(y.grad, want) and not y.grad[0, 0].any()
    y.grad = None
    a, h = d3.token_log_probs(y, t, entropy=True)
    assert torch.equal(h, H)
    h.sum().backward()                                  # the entropy alone
    want = d3.log_probs_grad(None, x, None, stats, entropy=H, dentropy=torch.ones(3, 4).cuda())
    assert torch.equal(y.grad, want)


def test_captured():
    g = torch.Generator().manual_seed(11)
    x, t = logits(g, 5, 40000, BF).cuda(), torch.randint(0, 40000, (5,), generator=g).cuda()
    gl = torch.randn(5, generator=g).cuda()
    d3.log_probs(x, t, entropy=True, top=9)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        got = d3.log_probs(x, t, entropy=True, top=9)
        dx = d3.log_probs_grad(gl, x, t, got[1])
    for k in range(4):
        x.copy_(logits(g, 5, 40000, BF))
        graph.replay()
        torch.cuda.synchronize()
        want = d3.log_probs(x, t, entropy=True, top=9)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(dx, d3.log_probs_grad(gl, x, t, want[1]))


def test_refusals():
    x, t = torch.zeros(4, 10, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    _, stats, H, _, _ = d3.log_probs(x, t, entropy=True)
    ones = torch.ones(4, device="cuda")
    for error, f in (
            (TypeError, lambda: d3.log_probs(x.double(), t)),
            (TypeError, lambda: d3.log_probs(x.cpu(), t)),
            (TypeError, lambda: d3.log_probs(x, t.float())),
            (TypeError, lambda: d3.log_probs(x, t.cpu())),
            (ValueError, lambda: d3.log_probs(x, t[:3])),
            (ValueError, lambda: d3.log_probs(x, t, top=11)),
            (ValueError, lambda: d3.log_probs(x, t, top=-1)),
            (ValueError, lambda: d3.log_probs(x.t(), t)),
            (d3.Dion3Error, lambda: d3.log_probs(torch.zeros(2, 99, device="cuda"), top=65)),
            (d3.Dion3Error, lambda: d3.log_probs(x, t, scale=0.0)),
            (d3.Dion3Error, lambda: d3.log_probs(x, t, scale=math.nan)),
            (ValueError, lambda: d3.log_probs_grad(None, x, t, stats)),
            (ValueError, lambda: d3.log_probs_grad(ones, x, None, stats)),
            (ValueError, lambda: d3.log_probs_grad(None, x, None, stats)),
            (ValueError, lambda: d3.log_probs_grad(ones, x, t, stats, dentropy=ones)),
            (ValueError, lambda: d3.log_probs_grad(ones, x, t, stats[:3])),
            (TypeError, lambda: d3.log_probs_grad(ones.double(), x, t, stats)),
            (TypeError, lambda: d3.log_probs_grad(ones, x, t, stats, out=x.half())),
            (ValueError, lambda: d3.log_probs_grad(ones, x, t, stats, out=x[:3]))):
        with pytest.raises(error):
            f()
