"""The layer operators against their formulas in 64 bits: norm with residual
and 8-bit output, linear products with epilogue, their gradients, the 8-bit
format.  Sizes are where the kernels change path: rows of one wave, of a
workgroup and longer; tiles' edges; split K; operands read in place and
copied; few tokens."""
import ctypes

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from orthogonalizing_optimizer_amd import _lib
from tests import layer_ref as ref
from tests.layer_ref import EPS32, U, close, d, rounded

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
DTYPES = [BF, FP]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def ints(g, *shape, most=4, dtype=BF):
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype)


def placed(t, how):
    """t on the GPU: contiguous, with a wider row stride (16-byte aligned or
    odd), or one element off alignment; what surrounds it is NaN."""
    if how == "plain":
        return t.cuda()
    T, m = t.shape
    ld, off = {"wide": (-(-m // 8) * 8 + 16, 8), "odd": (m + 3, 1), "off": (m, 1)}[how]
    buf = torch.full((T * ld + off + 64,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[off:off + T * ld].view(T, ld)[:, :m]
    v.copy_(t)
    return v


def same_bytes(got, want):
    """Equal e4m3 bytes; a NaN has two (either sign)."""
    got, want = (torch.where((b & 127) == 127, torch.full_like(b, 127), b) for b in (got.cpu(), want))
    return torch.equal(got, want)


# ------------------------------------------------------------------- the norm

# longest chain of additions behind a row's statistic: up to 32 terms in a
# thread (more in rows over 32768), 6 across the wave, 15 across waves
def chain(m):
    return 64 + 8 * (m // 8192)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m", [(1, 1), (1, 4096), (3, 7), (5, 32), (70, 100), (9, 512), (6, 515),
                                 (5, 1024), (130, 1030), (33, 2048), (4, 2049), (300, 4096),
                                 (3, 5120), (2, 8192), (2, 9001), (2, 16384), (2, 16390),
                                 (2, 32768), (2, 33001), (2, 70000)])
def test_add_rms_norm(T, m, dtype):
    g = gen(T * 131 + m)
    x, r = rnd(g, T, m, dtype=dtype), rnd(g, T, m, std=2.0, dtype=dtype)
    w = 1 + rnd(g, m, std=0.2)
    wt = w if m % 2 else w.to(dtype)
    y, h, rstd, p = d3.add_rms_norm(x.cuda(), wt.cuda(), residual=r.cuda(), eps=1e-5, pack=True)
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(dtype))
    hd = d(h)
    want = 1 / torch.sqrt((hd * hd).mean(1) + 1e-5)
    close(rstd, want, want * (chain(m) / 2 + 4) * EPS32, "rstd")
    yw = hd * want[:, None] * d(wt)
    close(y, yw, rounded(yw, dtype, yw.abs() * (chain(m) / 2 + 8) * EPS32), "y")
    q, s = ref.pack(y.cpu())
    assert torch.equal(p.scale.cpu(), s)
    assert torch.equal(p.q.view(torch.uint8).cpu(), q)
    # the parts one by one, with and without a residual
    y2, h2, _, none = d3.add_rms_norm(h, wt.cuda(), eps=1e-5)
    assert none is None and h2 is h and torch.equal(y2, y)
    none, _, _, p2 = d3.add_rms_norm(h, wt.cuda(), eps=1e-5, pack=True, return_y=False)
    assert none is None and torch.equal(p2.q.view(torch.uint8), p.q.view(torch.uint8))


@pytest.mark.parametrize("how", ["wide", "odd", "off"])
@pytest.mark.parametrize("m", [40, 333, 2500])
def test_add_rms_norm_places(m, how):
    g = gen(m)
    x, r, w = rnd(g, 9, m, dtype=BF), rnd(g, 9, m, dtype=BF), 1 + rnd(g, m, std=0.2)
    a = d3.add_rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), pack=True)
    b = d3.add_rms_norm(placed(x, how), w.cuda(), residual=placed(r, how), pack=True)
    for u, v in zip(a[:3], b[:3]):
        assert torch.equal(u, v)
    assert torch.equal(a[3].q.view(torch.uint8), b[3].q.view(torch.uint8))
    dy = rnd(g, 9, m, dtype=BF)
    ga = d3.add_rms_norm_grad(dy.cuda(), a[1], a[2], w.cuda(), dh=r.cuda())
    gb = d3.add_rms_norm_grad(placed(dy, how), placed(a[1].cpu(), how), a[2], w.cuda(),
                              dh=placed(r, how))
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])


def test_norm_row_without_values():
    """A row of zeros: y = 0 with eps, rstd = 1 / sqrt(eps); the gradient stays finite."""
    x = torch.zeros(3, 130, dtype=BF, device="cuda")
    x[1] = 1
    w = torch.ones(130, device="cuda")
    y, h, rstd, p = d3.add_rms_norm(x, w, eps=1e-6, pack=True)
    assert (y[0] == 0).all() and (y[2] == 0).all() and torch.isfinite(y).all()
    assert (p.scale[0] == 0).all() and (p.q.view(torch.uint8)[0] == 0).all()
    dx, dw = d3.add_rms_norm_grad(torch.ones_like(x), h, rstd, w)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m", [(1, 1), (1, 4096), (3, 7), (70, 100), (2100, 512), (6, 515),
                                 (5, 1024), (1500, 1030), (4, 2049), (1100, 4096), (3, 5120),
                                 (2, 9001), (2, 16384), (70, 16390), (2, 40000)])
def test_add_rms_norm_grad(T, m, dtype):
    g = gen(T * 7 + m)
    h, dy, dh = (rnd(g, T, m, dtype=dtype) for _ in range(3))
    w = 1 + rnd(g, m, std=0.2)
    rstd = (d(h).square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = d3.add_rms_norm_grad(dy.cuda(), h.cuda(), rstd.cuda(), w.cuda(), dh=dh.cuda())
    rs, u = d(rstd)[:, None], d(h) * d(rstd)[:, None]
    a = d(dy) * d(w)
    c = (a * u).mean(1, keepdim=True)
    want = rs * (a - u * c) + d(dh)
    size = rs * (a.abs() + u.abs() * (a * u).abs().mean(1, keepdim=True)) + d(dh).abs()
    close(dx, want, rounded(want, dtype, size * (chain(m) + 8) * EPS32), "dx")
    ww = (d(dy) * u).sum(0)
    # rows of a unit, the units of a slice, 64 slices
    close(dw, ww, (d(dy) * u).abs().sum(0) * (T + 4) * EPS32 + 1e-30, "dw")
    # no dh; one output alone
    dx2, none = d3.add_rms_norm_grad(dy.cuda(), h.cuda(), rstd.cuda(), w.cuda(), need_dw=False)
    assert none is None
    w2 = rs * (a - u * c)
    close(dx2, w2, rounded(w2, dtype, size * (chain(m) + 8) * EPS32), "dx without dh")
    none, dw2 = d3.add_rms_norm_grad(dy.cuda(), h.cuda(), rstd.cuda(), w.cuda(), need_dx=False)
    assert none is None and torch.equal(dw2, dw)


def test_norm_gradient_by_differences():
    """The gradient against central differences of the 64-bit formula."""
    g = gen(3)
    T, m = 3, 40
    h, dy, w = rnd(g, T, m, dtype=BF), rnd(g, T, m, dtype=BF), 1 + rnd(g, m, std=0.2)
    y, _, rstd, _ = d3.add_rms_norm(h.cuda(), w.cuda(), eps=1e-6)
    dx, dw = d3.add_rms_norm_grad(dy.cuda(), h.cuda(), rstd, w.cuda())

    def f(hh, ww):
        return (hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + 1e-6) * ww * d(dy)).sum()

    e = 1e-5
    for t in range(T):
        for j in range(0, m, 7):
            s = torch.zeros(T, m, dtype=torch.float64)
            s[t, j] = e
            num = (f(d(h) + s, d(w)) - f(d(h) - s, d(w))) / (2 * e)
            assert abs(float(dx[t, j]) - num) <= 2.0 ** -8 * abs(num) + 1e-6
    for j in range(0, m, 7):
        s = torch.zeros(m, dtype=torch.float64)
        s[j] = e
        num = (f(d(h), d(w) + s) - f(d(h), d(w) - s)) / (2 * e)
        assert abs(float(dw[j]) - num) <= 1e-6 * (1 + abs(num))


# ------------------------------------------------------------- 8-bit format

@pytest.mark.parametrize("dtype", [BF, FP, torch.float32])
@pytest.mark.parametrize("T,m", [(1, 1), (1, 32), (2, 33), (7, 31), (129, 100), (65, 4096), (3, 11008)])
def test_pack(T, m, dtype):
    g = gen(T + m)
    x = (torch.randn(T, m, generator=g) * torch.exp(3 * torch.randn(T, m, generator=g))).to(dtype)
    p = d3.pack_f8(x.cuda())
    q, s = ref.pack(x)
    assert torch.equal(p.scale.cpu(), s)
    assert same_bytes(p.q.view(torch.uint8), q)
    want = ref.unpack(q, s)[:, :m]
    for t in (BF, FP, torch.float32):
        y = d3.unpack_f8(p, t)
        # (an infinity among the fp16 inputs is a NaN in 8 bits)
        assert y.dtype == t and torch.equal(y.cpu().nan_to_num(3.0), want.to(t).nan_to_num(3.0))
        assert torch.equal(torch.isnan(y.cpu()), torch.isinf(x))
    # half a step of e4m3, or of its smallest step
    fin = torch.isfinite(x)
    err = (want - d(x)).abs()
    amax = torch.nn.functional.pad(torch.where(fin, d(x), 0.0), (0, (-m) % 32))
    amax = amax.view(T, -1, 32).abs().amax(2)
    small = (amax / 448 * 2 * 2.0 ** -10).repeat_interleave(32, 1)[:, :m]
    assert (err <= d(x).abs() * 2.0 ** -4 + small)[fin].all()


@pytest.mark.parametrize("how", ["wide", "odd", "off"])
def test_pack_places(how):
    x = rnd(gen(1), 11, 77, dtype=BF)
    a, b = d3.pack_f8(x.cuda()), d3.pack_f8(placed(x, how))
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
    assert torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("dtype", [BF, FP, torch.float32])
def test_pack_borders(dtype):
    """Zeros, infinities, NaN, the largest and smallest values, 448 and its neighbours, ties."""
    f = torch.finfo(dtype)
    rows = torch.zeros(9, 64)
    rows[1, 3], rows[1, 40] = float("inf"), float("nan")
    rows[1, 5] = 1.5
    rows[2, :32] = f.max
    rows[2, 32:] = -f.max
    rows[3, :] = torch.linspace(-f.max, f.max, 64)
    rows[4, 0], rows[4, 1] = f.tiny, -f.tiny / 2
    rows[5, 0], rows[5, 1], rows[5, 32] = 448.0, -447.0, 450.0
    rows[6, :32] = torch.arange(32) + 0.5
    rows[6, 32] = 448.0
    rows[6, 33:] = torch.arange(31) * 0.03125 + 17.0
    rows[7, 0] = float("-inf")
    rows[8, 0], rows[8, 33] = f.smallest_normal * f.eps, -0.0
    x = rows.to(dtype)
    p = d3.pack_f8(x.cuda())
    q, s = ref.pack(x)
    assert torch.equal(p.scale.cpu(), s)
    assert same_bytes(p.q.view(torch.uint8), q)
    y = d3.unpack_f8(p, dtype).cpu()
    assert torch.isfinite(y[torch.isfinite(x)]).all()
    assert torch.isnan(y[~torch.isfinite(x)]).all()


@pytest.mark.parametrize("t", [BF, FP, torch.float32])
def test_unpack_every_byte(t):
    """Every e4m3 byte under every scale, rounded once to the type."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 8).contiguous()
    s = s.clamp_max(247)                    # the scales that a block can take
    p = d3.PackedF8(q.cuda().view(torch.float8_e4m3fn), s.cuda(), 256)
    y = d3.unpack_f8(p, t).cpu()
    want = ref.unpack(q, s)
    tiny = want.abs() < torch.finfo(t).tiny
    over = want.abs() > torch.finfo(t).max
    nan = torch.isnan(want)
    ok = ~(tiny | over | nan)
    assert torch.equal(y[ok], want.to(t)[ok])
    assert torch.isnan(y[nan]).all()
    close(y[tiny], want[tiny], torch.full_like(want[tiny], torch.finfo(t).tiny * torch.finfo(t).eps))


# ------------------------------------------------------------------ products

SHAPES = [(1, 1, 1), (1, 16, 8), (2, 15, 9), (5, 100, 130), (16, 17, 1024), (17, 16, 64),
          (1, 520, 4104), (33, 130, 72), (64, 128, 64), (128, 128, 192), (129, 127, 200),
          (200, 300, 515), (257, 256, 128), (300, 520, 1000), (1000, 264, 320), (513, 1030, 96)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,m", SHAPES)
def test_products_exact(T, n, m, dtype):
    """Small whole numbers: every product and sum is exact in fp32 (at most
    1030 * 16 + bias < 2^24), so each output is the exact value rounded once."""
    g = gen(T + 31 * n + 17 * m)
    x, w, dz = ints(g, T, m, dtype=dtype), ints(g, n, m, dtype=dtype), ints(g, T, n, dtype=dtype)
    b, r, rx = ints(g, n, dtype=torch.float32), ints(g, T, n, dtype=dtype), ints(g, T, m, dtype=dtype)
    y, z = d3.linear(x.cuda(), w.cuda(), bias=b.cuda(), residual=r.cuda(), act="relu",
                     return_preact=True)
    zw = d(x) @ d(w).T + d(b)
    assert torch.equal(z.cpu(), zw.to(dtype))
    assert torch.equal(y.cpu(), (zw.clamp_min(0) + d(r)).to(dtype))
    y, z = d3.linear(x.cuda(), w.cuda())
    assert z is None and torch.equal(y.cpu(), (d(x) @ d(w).T).to(dtype))
    dxw = d(dz) @ d(w)
    assert torch.equal(d3.linear_grad_input(dz.cuda(), w.cuda()).cpu(), dxw.to(dtype))
    assert torch.equal(d3.linear_grad_input(dz.cuda(), w.cuda(), residual=rx.cuda()).cpu(),
                       (dxw + d(rx)).to(dtype))
    gw = d(dz).T @ d(x)
    out = d3.linear_grad_weight(dz.cuda(), x.cuda())
    assert out.dtype == torch.float32 and torch.equal(d(out), gw)
    assert torch.equal(d(d3.linear_grad_weight(dz.cuda(), x.cuda(), out=out, accumulate=True)), 2 * gw)
    assert torch.equal(d(d3.linear_grad_weight(dz.cuda(), x.cuda(), out=out)), gw)
    p = d3.pack_f8(x.cuda())                       # (whole numbers up to 4 are exact in 8 bits)
    assert torch.equal(d(d3.linear_grad_weight(dz.cuda(), p)), gw)
    assert torch.equal(d(d3.linear_grad_weight(dz.cuda(), p, out=out, accumulate=True)), 2 * gw)


@pytest.mark.parametrize("T,n,m", [(2100, 4100, 72), (4100, 2120, 40), (2100, 72, 4100),
                                   (4200, 40, 2100), (72, 2100, 4100), (40, 4200, 2150),
                                   (3000, 6300, 64)])
def test_products_of_many_tiles(T, n, m):
    """More tiles than one round of workgroups, with a remainder: the output is
    cut in two rectangles, by rows or by columns, each exact."""
    test_products_exact(T, n, m, BF)


@pytest.mark.parametrize("how", ["odd", "off"])
@pytest.mark.parametrize("T,n,m", [(2100, 4101, 77), (4101, 2123, 45), (77, 4103, 4101),
                                   (2101, 77, 4100), (3001, 6301, 70), (1000, 1029, 5121),
                                   (2048, 8193, 1001), (2048, 1001, 8193), (700, 8, 9), (9, 700, 8), (8, 9, 700), (300, 7, 5), (130, 66, 17)])
def test_ragged_products(T, n, m, how):
    """Unaligned operands read as they are, by every tile that does so, with
    odd ends along K and along both sides, parts of the output and of K."""
    test_products_places(T, n, m, how)


@pytest.mark.parametrize("how", ["wide", "odd", "off"])
@pytest.mark.parametrize("T,n,m", [(3, 40, 72), (5, 33, 101), (150, 264, 136), (141, 131, 203),
                                   (300, 257, 520)])
def test_products_places(T, n, m, how):
    """Row strides and alignments, with NaN all round the operands."""
    g = gen(T + n + m)
    x, w, dz = ints(g, T, m), ints(g, n, m), ints(g, T, n)
    r = ints(g, T, n)
    X, W, Z, R = (placed(t, how) for t in (x, w, dz, r))
    y, _ = d3.linear(X, W, residual=R)
    assert torch.equal(y.cpu(), (d(x) @ d(w).T + d(r)).to(BF))
    assert torch.equal(d3.linear_grad_input(Z, W).cpu(), (d(dz) @ d(w)).to(BF))
    out = placed(torch.ones(n, m), "wide" if how == "wide" else "odd")
    whole = out._base.clone()
    got = d3.linear_grad_weight(Z, X, out=out, accumulate=True)
    assert got.data_ptr() == out.data_ptr() and torch.equal(d(out), d(dz).T @ d(x) + 1)
    out.copy_(torch.ones(n, m))
    assert torch.equal(out._base.view(torch.int32), whole.view(torch.int32))   # nothing else written
    # mixed: one operand in place, the other copied
    assert torch.equal(d3.linear(x.cuda(), W)[0].cpu(), (d(x) @ d(w).T).to(BF))
    assert torch.equal(d(d3.linear_grad_weight(Z, x.cuda())), d(dz).T @ d(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,n,m", [(1, 200, 328), (40, 136, 203), (300, 260, 512)])
def test_linear_values(T, n, m, act, dtype):
    g = gen(T + n)
    x, w = rnd(g, T, m, std=2.0, dtype=dtype), rnd(g, n, m, std=0.1, dtype=dtype)
    b = rnd(g, n, dtype=dtype)
    r = rnd(g, T, n, dtype=dtype)
    y, z = d3.linear(x.cuda(), w.cuda(), bias=b.cuda(), act=act, residual=r.cuda(),
                     return_preact=True)
    zw = d(x) @ d(w).T + d(b)
    dzw = (d(x).abs() @ d(w).abs().T + d(b).abs()) * (m + 4) * EPS32
    close(z, zw, rounded(zw, dtype, dzw), "z")
    aw = ref.act(zw, act)
    # |act'| <= 1.13
    ea = 1.13 * dzw + zw.abs() * ref.ACT_EPS + d(r).abs() * EPS32 + aw.abs() * EPS32
    close(y, aw + d(r), rounded(aw + d(r), dtype, ea), "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,m", [(16384, 128, 512), (4100, 100, 40), (700, 600, 264)])
def test_grad_weight_values(T, n, m, dtype):
    g = gen(T)
    dz, x, M = rnd(g, T, n, std=0.05, dtype=dtype), rnd(g, T, m, dtype=dtype), rnd(g, n, m)
    p = d3.pack_f8(x.cuda())
    xq = d3.unpack_f8(p, torch.float32).cpu()
    for xs, xv in ((x.cuda(), x), (p, xq)):
        out = M.cuda()
        d3.linear_grad_weight(dz.cuda(), xs, out=out, accumulate=True)
        want = d(dz).T @ d(xv) + d(M)
        size = d(dz).abs().T @ d(xv).abs() + d(M).abs()
        close(out, want, size * (T + 4) * EPS32, "M")
        # far closer on average than that: a root of the chain's length
        assert (d(out) - want).norm() <= 4 * EPS32 * T ** 0.5 * size.norm()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,n", [(1, 1), (3, 33), (40, 515), (700, 1032), (5000, 70)])
def test_act_grad(T, n, act, dtype):
    g = gen(T + n)
    dy, z = rnd(g, T, n, dtype=dtype), rnd(g, T, n, std=3.0, dtype=dtype)
    zp = d3.pack_f8(z.cuda())
    for zs, zv in ((z.cuda(), z), (zp, d3.unpack_f8(zp, torch.float32).cpu())):
        dz, db = d3.act_grad(dy.cuda(), zs, act, bias=True)
        v = d(dy) * ref.act_slope(d(zv), act)
        e = d(dy).abs() * (1 + d(zv).abs()) * ref.ACT_EPS if act != "none" else 0 * d(dy)
        close(dz, v, rounded(v, dtype, e), "dz")
        close(db, v.sum(0), e.sum(0) + (v.abs() + e).sum(0) * (T + 1) * EPS32 + 1e-30, "db")
        dz2, none = d3.act_grad(dy.cuda(), zs, act)
        assert none is None and torch.equal(dz2, dz)


@pytest.mark.parametrize("act", ACTS)
def test_act_gradient_by_differences(act):
    z = torch.tensor([[-6.0, -2.5, -0.75, -0.125, 0.25, 0.5, 1.5, 4.0]], dtype=BF)
    dz, _ = d3.act_grad(torch.ones_like(z).cuda(), z.cuda(), act)
    e = 1e-6
    num = (ref.act(d(z) + e, act) - ref.act(d(z) - e, act)) / (2 * e)
    close(dz, num, num.abs() * U[BF] + 1e-6)


# ------------------------------------------------------- ends of the ranges

def test_no_tokens():
    for lead in [(0,), (2, 0), (0, 3)]:
        x = torch.empty(*lead, 40, dtype=BF, device="cuda")
        w = torch.ones(24, 40, dtype=BF, device="cuda")
        dz = torch.empty(*lead, 24, dtype=BF, device="cuda")
        y, z = d3.linear(x, w, return_preact=True)
        assert y.shape == z.shape == torch.Size((*lead, 24))
        assert d3.linear_grad_input(dz, w).shape == x.shape
        p = d3.pack_f8(x)
        assert d3.unpack_f8(p).shape == x.shape
        for xs in (x, p):
            out = torch.full((24, 40), 3.0, device="cuda")
            assert (d3.linear_grad_weight(dz, xs, out=out, accumulate=True) == 3).all()
            assert (d3.linear_grad_weight(dz, xs, out=out) == 0).all()
        yn, h, rstd, pk = d3.add_rms_norm(x, torch.ones(40, device="cuda"), residual=x, pack=True)
        assert yn.shape == h.shape == x.shape and pk.rows == 0
        dx, dw = d3.add_rms_norm_grad(x, x, rstd, torch.ones(40, device="cuda"))
        assert dx.shape == x.shape and (dw == 0).all()
        dzz, db = d3.act_grad(dz, dz, "silu", bias=True)
        assert dzz.shape == dz.shape and (db == 0).all()


def test_leading_dimensions():
    g = gen(2)
    x, w = ints(g, 3, 5, 64), ints(g, 40, 64)
    dz = ints(g, 3, 5, 40)
    y, _ = d3.linear(x.cuda(), w.cuda())
    assert y.shape == (3, 5, 40) and torch.equal(y.cpu(), (d(x) @ d(w).T).to(BF))
    gw = d(dz).reshape(15, 40).T @ d(x).reshape(15, 64)
    assert torch.equal(d(d3.linear_grad_weight(dz.cuda(), x.cuda())), gw)
    assert torch.equal(d(d3.linear_grad_weight(dz.cuda(), d3.pack_f8(x.cuda()))), gw)
    # a slice of the features of a wider tensor: one stride for all rows
    wide = torch.full((3, 5, 100), float("nan"), dtype=BF, device="cuda")
    wide[..., 8:72] = x.cuda()
    assert torch.equal(d3.linear(wide[..., 8:72], w.cuda())[0], y)
    with pytest.raises(ValueError):
        d3.linear(torch.zeros(5, 3, 64, dtype=BF, device="cuda").transpose(0, 1), w.cuda())


def test_offsets_past_32_bits():
    """Operands beyond 2^32 bytes: rows at their ends count, and the right ones."""
    T, n, m = 300_001, 8192, 64
    dz = torch.zeros(T, n, dtype=BF, device="cuda")
    x = torch.zeros(T, m, dtype=BF, device="cuda")
    rows = [0, 131_071, 131_072, 262_144, T - 1]
    g = gen(9)
    a, b = ints(g, len(rows), n), ints(g, len(rows), m)
    dz[rows], x[rows] = a.cuda(), b.cuda()
    want = d(a).T @ d(b)
    assert torch.equal(d(d3.linear_grad_weight(dz, x)), want)
    assert torch.equal(d(d3.linear_grad_weight(dz, d3.pack_f8(x))), want)
    w = ints(g, n, m)
    dx = d3.linear_grad_input(dz, w.cuda())
    assert torch.equal(dx[rows].cpu(), (d(a) @ d(w)).to(BF))
    assert int((dx != 0).any(1).sum()) <= len(rows)
    y, _ = d3.linear(x, w.cuda())                              # output past 2^32 bytes
    assert torch.equal(y[rows].cpu(), (d(b) @ d(w).T).to(BF))
    y.zero_()
    y[rows] = a.cuda()
    p = d3.pack_f8(y)                                           # 8-bit data past 2^31
    q, s = ref.pack(a)
    assert torch.equal(p.q[rows].view(torch.uint8).cpu(), q) and torch.equal(p.scale[rows].cpu(), s)
    assert torch.equal(d3.unpack_f8(p)[rows], y[rows])
    dzz, db = d3.act_grad(y, p, "relu", bias=True)
    assert torch.equal(d(db), d(a).clamp_min(0).sum(0))
    h = y
    yn, _, rstd, _ = d3.add_rms_norm(h, torch.ones(n, device="cuda"))
    small = d3.add_rms_norm(h[rows].contiguous(), torch.ones(n, device="cuda"))
    assert torch.equal(yn[rows], small[0]) and torch.equal(rstd[rows], small[2])
    dx, dw = d3.add_rms_norm_grad(h, h, rstd, torch.ones(n, device="cuda"))
    dxs, dws = d3.add_rms_norm_grad(h[rows].contiguous(), h[rows].contiguous(), small[2],
                                    torch.ones(n, device="cuda"))
    assert torch.equal(dx[rows], dxs)
    close(dw, d(dws), d(dws).abs() * 16 * EPS32 + 1e-30)


# ---------------------------------------------------- C calls, streams, graphs

def test_c_call_writes_its_rows_only():
    """Outputs with wide rows: what lies between and behind them is left as it was."""
    T, n, m = 37, 41, 72
    g = gen(4)
    x, w = ints(g, T, m).cuda(), ints(g, n, m).cuda()
    Y = torch.full((T + 2, n + 9), 7.0, dtype=BF, device="cuda")
    Z = torch.full((T + 2, n + 9), 7.0, dtype=BF, device="cuda")
    nb = ctypes.c_size_t()
    lib = d3.lib()
    assert lib.dion3_linear_workspace_size(x.data_ptr(), m, w.data_ptr(), m, T, n, m,
                                           ctypes.byref(nb)) == 0
    ws = torch.empty(nb.value + 256, dtype=torch.uint8, device="cuda")
    p = ws.data_ptr() + (-ws.data_ptr()) % 256
    s = torch.cuda.current_stream().cuda_stream
    assert lib.dion3_linear(x.data_ptr(), m, w.data_ptr(), m, None, 0, None, 0, Y.data_ptr(), n + 9,
                            Z.data_ptr(), n + 9, T, n, m, 0, 1, p, nb.value, s) == 0
    want = (d(x) @ d(w).T).to(BF)
    for o in (Y, Z):
        assert torch.equal(o[:T, :n].cpu(), want)
        assert (o[T:] == 7).all() and (o[:, n:] == 7).all()


def _all(x, r, w, nw, dy, M):
    """One pass of every operator, as a layer runs them."""
    y, h, rstd, p = d3.add_rms_norm(x, nw, residual=r, pack=True)
    o, z = d3.linear(y, w, act="gelu_tanh", return_preact=True)
    zp = d3.pack_f8(z)
    dz, db = d3.act_grad(dy, zp, "gelu_tanh", bias=True)
    dyn = d3.linear_grad_input(dz, w)
    d3.linear_grad_weight(dz, p, out=M, accumulate=True)
    dx, dnw = d3.add_rms_norm_grad(dyn, h, rstd, nw, dh=r)
    return [y, h, rstd, o, z, dz, db, dyn, dx, dnw, M]


def _inputs(seed, T=200, n=520, m=264):
    g = gen(seed)
    return [t.cuda() for t in (rnd(g, T, m, dtype=BF), rnd(g, T, m, dtype=BF),
                               rnd(g, n, m, std=0.05, dtype=BF), 1 + rnd(g, m, std=0.1),
                               rnd(g, T, n, dtype=BF), rnd(g, n, m))]


def test_same_bits_every_time():
    a = [t.clone() for t in _all(*_inputs(1))]
    for _ in range(3):
        for u, v in zip(a, _all(*_inputs(1))):
            assert torch.equal(u, v)


def test_two_streams():
    """Calls in flight on two streams share nothing."""
    want = [[t.clone() for t in _all(*_inputs(s, T=3000))] for s in (1, 2)]
    ins = [_inputs(s, T=3000) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, i in zip(streams, ins):
        with torch.cuda.stream(s):
            got.append(_all(*i))
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        for u, v in zip(w, o):
            assert torch.equal(u, v)


@pytest.mark.parametrize("T,n,m", [(200, 520, 264), (1, 100, 130), (2048, 128, 512)])
def test_graphs(T, n, m):
    """Two captured graphs, replayed in turn with eager work between: every
    replay equals the eager result."""
    seeds = (5, 6)
    want = [[t.clone() for t in _all(*_inputs(s, T, n, m))] for s in seeds]
    ins = [_inputs(s, T, n, m) for s in seeds]
    M0 = [i[5].clone() for i in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in ins:
            _all(*i)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for i in ins:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_all(*i))
        graphs.append(gr)
    for rep in range(3):
        for k in (0, 1):
            ins[k][5].copy_(M0[k])
            graphs[k].replay()
        _all(*_inputs(9, T, n, m))
        torch.cuda.synchronize()
        for k in (0, 1):
            for u, v in zip(want[k], outs[k]):
                assert torch.equal(u, v), (rep, k)


def test_user_workspace():
    ws = _lib.Workspace()
    g = gen(8)
    dz, x = ints(g, 5000, 100), ints(g, 5000, 60)
    for T in (10, 5000, 700):
        assert torch.equal(d(d3.linear_grad_weight(dz[:T].cuda(), x[:T].cuda(), ws=ws)),
                           d(dz[:T]).T @ d(x[:T]))
