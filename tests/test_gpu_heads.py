"""Norms of queries and keys with the rotation against the formulas in 64 bits:
head sizes around the lanes' pieces, both orders of pairs, partly turned heads,
far positions, layouts, gradients.

Bounds: the statistic goes through at most 16 additions in a lane and 6 across
lanes; an angle is reduced in 64 bits, its turn rounded to fp32 (pi 2^-24 of an
angle of at most pi), sine and cosine off by 4 EPS32 more."""
import math

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, close, d, rounded

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
CHAIN, TURN = 24, 8
# T, query heads, key heads, columns, turned columns
SIZES = [(1, 1, 0, 8, 8), (1, 32, 8, 128, 128), (3, 2, 1, 64, 64), (5, 3, 3, 80, 20), (7, 5, 2, 96, 48),
         (300, 16, 4, 128, 128), (4, 2, 2, 256, 64), (3, 1, 1, 1, 0), (3, 2, 2, 7, 4), (2, 3, 1, 5, 2),
         (6, 70, 3, 33, 30), (2, 1, 2, 512, 512), (2, 1, 1, 1024, 1024), (9, 4, 2, 1000, 500),
         (4500, 3, 1, 48, 16), (0, 4, 2, 64, 32), (5, 2, 1, 40, 0)]


def rnd(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def freqs_of(r, base=10000.0):
    return base ** (-torch.arange(0, r, 2, dtype=torch.float64) / max(r, 1))


def turn(x, pos, freqs, interleaved, sign=1.0):
    """x [..., H, D] in 64 bits, turned."""
    h = freqs.shape[0]
    a = (pos.double()[..., None] * freqs)[..., None, :]
    c, s = torch.cos(a), sign * torch.sin(a)
    y = x.clone()
    u, v = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    if interleaved:
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = u * c - v * s, v * c + u * s
    else:
        y[..., :h], y[..., h:2 * h] = u * c - v * s, v * c + u * s
    return y


def partner(x, freqs, interleaved):
    """|x| plus the magnitude of the other member of each pair."""
    h = freqs.shape[0]
    x = x.abs()
    o = torch.zeros_like(x)
    if interleaved:
        o[..., 0:2 * h:2], o[..., 1:2 * h:2] = x[..., 1:2 * h:2], x[..., 0:2 * h:2]
    else:
        o[..., :h], o[..., h:2 * h] = x[..., h:2 * h], x[..., :h]
    return x + o


def formula(x, w, pos, freqs, interleaved, eps):
    x, w = d(x), d(w)
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = x * rstd * w
    return turn(u, pos, freqs, interleaved), partner(u, freqs, interleaved)


def grad_formula(dy, x, w, pos, freqs, interleaved, eps):
    """dx, dw and what their bounds scale with."""
    dy, x, w = d(dy), d(x), d(w)
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    hat, du = x * rstd, turn(dy, pos, freqs, interleaved, -1.0)
    size = partner(dy, freqs, interleaved)
    a = du * w
    dx = rstd * (a - hat * (a * hat).mean(-1, keepdim=True))
    lim = rstd * (size * w.abs() + hat.abs() * (size * w.abs() * hat.abs()).mean(-1, keepdim=True))
    dims = tuple(range(x.dim() - 1))
    return dx, lim, (du * hat).sum(dims), (size * hat.abs()).sum(dims)


def inputs(g, T, hq, hk, D, r, dtype, wtype):
    q, k = rnd(g, T, hq, D, dtype=dtype), rnd(g, T, max(hk, 1), D, dtype=dtype, std=3.0)
    wq, wk = ((1 + 0.2 * rnd(g, D)).to(wtype) for _ in range(2))
    return q, k, wq, wk, freqs_of(r)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,hq,hk,D,r", SIZES)
def test_forward_and_gradient(T, hq, hk, D, r, dtype, interleaved):
    g = torch.Generator().manual_seed(T + 7 * D + r)
    wtype = dtype if D % 16 == 0 else torch.float32
    q, k, wq, wk, fr = inputs(g, T, hq, hk, D, r, dtype, wtype)
    pos = torch.randint(-50, 5000, (T,), generator=g)
    pos = pos.int() if hq % 2 else pos
    eps = 1e-5
    kc, wkc = (k.cuda(), wk.cuda()) if hk else (None, None)
    args = (q.cuda(), kc, wq.cuda(), wkc, pos.cuda(), fr.cuda())
    yq, yk = d3.qk_norm_rope(*args, eps=eps, interleaved=interleaved)
    assert (yk is None) == (hk == 0)
    dyq, dyk = rnd(g, T, hq, D, dtype=dtype), rnd(g, T, max(hk, 1), D, dtype=dtype)
    dq, dk, dwq, dwk = d3.qk_norm_rope_grad(dyq.cuda(), dyk.cuda() if hk else None, *args, eps=eps,
                                            interleaved=interleaved)
    assert (dk is None) == (hk == 0) and (dwk is None) == (hk == 0)
    for x, w, y, dy, dx, dw in ((q, wq, yq, dyq, dq, dwq), (k, wk, yk, dyk, dk, dwk))[:1 + (hk > 0)]:
        want, size = formula(x, w, pos, fr, interleaved, eps)
        close(y, want, rounded(want, dtype, size * (CHAIN / 2 + TURN + 4) * EPS32), "y")
        wx, lim, ww, wl = grad_formula(dy, x, w, pos, fr, interleaved, eps)
        close(dx, wx, rounded(wx, dtype, lim * (2 * CHAIN + TURN + 8) * EPS32), "dx")
        n = x.shape[0] * x.shape[1]
        close(dw, ww, wl * (n + CHAIN + TURN) * EPS32 + 1e-30, "dw")
    again = d3.qk_norm_rope_grad(dyq.cuda(), dyk.cuda() if hk else None, *args, eps=eps,
                                 interleaved=interleaved, need_dw=False)
    assert torch.equal(again[0], dq) and again[2] is None and again[3] is None
    again = d3.qk_norm_rope_grad(dyq.cuda(), dyk.cuda() if hk else None, *args, eps=eps,
                                 interleaved=interleaved, need_dx=False)
    assert again[0] is None and torch.equal(again[2], dwq)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [100000, 1 << 24, -(1 << 30), (1 << 40) + 3])
def test_far_positions(far, interleaved):
    """A frequency of 1 at a far position: the angle keeps its bits.  The
    reference's own angle is off by half a step of 64 bits."""
    g = torch.Generator().manual_seed(1)
    T, D = 33, 128
    q, k, wq, wk, fr = inputs(g, T, 2, 1, D, D, BF, torch.float32)
    pos = far + torch.arange(T)
    yq, yk = d3.qk_norm_rope(q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), pos.cuda(), fr.cuda(),
                             interleaved=interleaved)
    for x, w, y in ((q, wq, yq), (k, wk, yk)):
        want, size = formula(x, w, pos, fr, interleaved, 1e-6)
        angle = abs(far) * 4 * 2.0 ** -53
        close(y, want, rounded(want, BF, size * ((CHAIN / 2 + TURN + 4) * EPS32 + angle)))


def views(t, how):
    """t [B, S, H, D] in another layout of the same values, NaN around it."""
    B, S, H, D = t.shape
    if how == "packed":                          # between other columns of one product
        buf = torch.full((B, S, (H + 3) * D + 5), float("nan"), dtype=t.dtype, device="cuda")
        v = buf[..., D + 1:D + 1 + H * D].unflatten(-1, (H, D))
    elif how == "heads first":                   # [H, B S, D]
        v = torch.empty(H, B * S, D, dtype=t.dtype, device="cuda").transpose(0, 1)
        v = v.unflatten(0, (B, S))
    else:
        buf = torch.full((t.numel() + 9,), float("nan"), dtype=t.dtype, device="cuda")
        v = buf[3:3 + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("how", ["packed", "heads first", "off"])
@pytest.mark.parametrize("D,r", [(128, 128), (80, 20), (7, 6)])
def test_layouts(D, r, how):
    g = torch.Generator().manual_seed(D)
    B, S, hq, hk = 2, 17, 6, 2
    q, k = rnd(g, B, S, hq, D, dtype=BF).cuda(), rnd(g, B, S, hk, D, dtype=BF).cuda()
    dyq, dyk = rnd(g, B, S, hq, D, dtype=BF).cuda(), rnd(g, B, S, hk, D, dtype=BF).cuda()
    w = (1 + 0.1 * rnd(g, D)).cuda()
    fr, pos = freqs_of(r).cuda(), torch.arange(S, device="cuda")       # shared by the batch
    a = d3.qk_norm_rope(q, k, w, w, pos, fr)
    b = d3.qk_norm_rope(views(q, how), views(k, how), w, w, pos.expand(B, S), fr)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert b[0].is_contiguous() and b[0].shape == (B, S, hq, D)
    ga = d3.qk_norm_rope_grad(dyq, dyk, q, k, w, w, pos, fr)
    gb = d3.qk_norm_rope_grad(views(dyq, how), views(dyk, how), views(q, how), views(k, how), w, w,
                              pos, fr)
    for u, v in zip(ga, gb):
        assert torch.equal(u, v)


def test_rows_without_values():
    """A head of zeros stays zeros, its gradient finite; infinities and NaN stay in their heads."""
    q = torch.ones(2, 4, 64, dtype=BF, device="cuda")
    q[0, 1] = 0
    q[1, 2, 5] = float("nan")
    q[1, 3, 60] = float("inf")
    w, fr, pos = torch.ones(64, device="cuda"), freqs_of(32).cuda(), torch.arange(2, device="cuda")
    y, _ = d3.qk_norm_rope(q, None, w, None, pos, fr)
    dq, _, dw, _ = d3.qk_norm_rope_grad(torch.ones_like(q), None, q, None, w, None, pos, fr)
    assert not y[0, 1].any() and torch.isfinite(dq[0]).all()
    assert torch.isnan(y[1, 2]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[1, :2]).all()
    # 1 / sqrt(inf) = 0: only the infinity itself is NaN, past the turned columns
    assert torch.isnan(y[1, 3, 60]) and int(torch.isnan(y[1, 3]).sum()) == 1


def test_gradient_by_differences():
    g = torch.Generator().manual_seed(5)
    T, H, D, r = 2, 2, 24, 16
    q, dy = rnd(g, T, H, D, dtype=BF), rnd(g, T, H, D, dtype=BF)
    w, pos, fr = 1 + 0.2 * rnd(g, D), torch.tensor([3, 1000]), freqs_of(r)
    dq, _, dw, _ = d3.qk_norm_rope_grad(dy.cuda(), None, q.cuda(), None, w.cuda(), None, pos.cuda(),
                                        fr.cuda())

    def f(x, ww):
        rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        return (turn(x * rstd * ww, pos, fr, False) * d(dy)).sum()

    e = 1e-5
    for t, h, j in ((0, 0, 0), (0, 1, 9), (1, 0, 15), (1, 1, 16), (1, 0, 23)):
        s = torch.zeros(T, H, D, dtype=torch.float64)
        s[t, h, j] = e
        num = float(f(d(q) + s, d(w)) - f(d(q) - s, d(w))) / (2 * e)
        assert abs(float(dq[t, h, j]) - num) <= 2.0 ** -8 * abs(num) + 1e-5
    for j in range(0, D, 5):
        s = torch.zeros(D, dtype=torch.float64)
        s[j] = e
        num = float(f(d(q), d(w) + s) - f(d(q), d(w) - s)) / (2 * e)
        assert abs(float(dw[j]) - num) <= 1e-5 * (1 + abs(num))


@pytest.mark.parametrize("wtype", [BF, torch.float32])
def test_differentiable_form(wtype):
    """The operators' own gradients, for what asks for one; either output alone."""
    g = torch.Generator().manual_seed(6)
    B, S, hq, hk, D = 2, 9, 4, 2, 32
    x = rnd(g, B, S, (hq + 2 * hk) * D, dtype=BF).cuda().requires_grad_(True)
    wq, wk = ((1 + 0.1 * rnd(g, D)).to(wtype).cuda().requires_grad_(True) for _ in range(2))
    pos, fr = torch.arange(S, device="cuda"), freqs_of(D).cuda()

    def split(t):
        return t[..., :hq * D].unflatten(-1, (hq, D)), t[..., hq * D:(hq + hk) * D].unflatten(-1, (hk, D))

    dyq, dyk = rnd(g, B, hq, S, D, dtype=BF).cuda(), rnd(g, B, hk, S, D, dtype=BF).cuda()
    q, k = split(x)
    yq, yk = d3.qk_norm_rope_layer(q, k, wq, wk, pos, fr)
    # gradients as attention hands them back: heads before tokens
    torch.autograd.backward([yq, yk], [dyq.transpose(1, 2), dyk.transpose(1, 2)])
    q, k = split(x.detach())
    want = d3.qk_norm_rope_grad(dyq.transpose(1, 2).contiguous(), dyk.transpose(1, 2).contiguous(), q, k,
                                wq.detach(), wk.detach(), pos, fr)
    gq, gk = split(x.grad)
    assert torch.equal(gq, want[0]) and torch.equal(gk, want[1])
    assert not x.grad[..., (hq + hk) * D:].any()
    assert torch.equal(wq.grad, want[2].to(wtype)) and torch.equal(wk.grad, want[3].to(wtype))
    x.grad = wq.grad = wk.grad = None
    yq, yk = d3.qk_norm_rope_layer(*split(x), wq, wk, pos, fr)
    yk.backward(dyk.transpose(1, 2))                    # keys alone
    assert torch.equal(split(x.grad)[1], want[1]) and not split(x.grad)[0].any()
    # (the order of the weights' sums goes by the sizes, those of a call without queries here)
    alone = d3.qk_norm_rope_grad(dyk.transpose(1, 2).contiguous(), None, k, None, wk.detach(), None, pos, fr)
    assert wq.grad is None and torch.equal(wk.grad, alone[2].to(wtype))
    x.grad = None
    yq, none = d3.qk_norm_rope_layer(split(x)[0], None, wq.detach(), None, pos, fr)
    yq.sum().backward()                                 # queries alone, an expanded gradient
    assert none is None and torch.isfinite(x.grad).all()


def test_in_place_and_captured():
    """Y over X (and dX over dY) through the C interface, in a captured graph."""
    import ctypes
    from orthogonalizing_optimizer_amd import _lib
    g = torch.Generator().manual_seed(7)
    T, H, D = 37, 5, 96
    src = rnd(g, T, H, D, dtype=BF).cuda()
    x, w, fr, pos = src.clone(), torch.ones(D, device="cuda"), freqs_of(64).cuda(), torch.arange(T, device="cuda")
    want, _ = d3.qk_norm_rope(src, None, w, None, pos, fr)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        desc = _lib.HeadsDesc(X=x.data_ptr(), ldx=H * D, hsx=D, w=w.data_ptr(), Y=x.data_ptr(),
                              ldy=H * D, hsy=D, heads=H)
        st = d3.lib().dion3_qk_norm_rope(ctypes.byref(desc), None, fr.data_ptr(), pos.data_ptr(), 64, T,
                                         D, 64, 0, 1e-6, 0, 1, torch.cuda.current_stream().cuda_stream)
        y2, _ = d3.qk_norm_rope(src, None, w, None, pos, fr)
        grads = d3.qk_norm_rope_grad(y2, None, src, None, w, None, pos, fr)
    assert st == 0
    for _ in range(3):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want) and torch.equal(y2, want)
        eager = d3.qk_norm_rope_grad(want, None, src, None, w, None, pos, fr)
        assert torch.equal(grads[0], eager[0]) and torch.equal(grads[2], eager[2])


@pytest.mark.parametrize("heads", [1, 2, 3, 20])
@pytest.mark.parametrize("D,r,interleaved", [(80, 20, False), (96, 24, True), (9, 0, False), (17, 8, True),
                                             (26, 18, False), (100, 50, False), (112, 112, False),
                                             (23, 6, False), (8, 8, True), (16, 16, False), (64, 10, True),
                                             (72, 16, False), (1000, 24, False), (130, 130, True)])
def test_over_the_inputs(D, r, interleaved, heads):
    """Y over X and dX over dY or X, where chunks of columns lie over each
    other, end early or fit, and batches hold one token or several."""
    import ctypes
    from orthogonalizing_optimizer_amd import _lib
    g = torch.Generator().manual_seed(D + r)
    T, ld = 53, heads * D + 3
    x, dy = (rnd(g, T, heads, D, dtype=BF).cuda() for _ in range(2))
    w, fr = rnd(g, D).cuda(), freqs_of(r).cuda()
    pos = torch.randint(0, 3000, (T,), generator=g).cuda()
    y, _ = d3.qk_norm_rope(x, None, w, None, pos, fr, interleaved=interleaved)
    want, _, wdw, _ = d3.qk_norm_rope_grad(dy, None, x, None, w, None, pos, fr, interleaved=interleaved)

    def laid(t):
        buf = torch.full((T * ld + 8,), 7.0, dtype=BF, device="cuda")
        v = buf.as_strided((T, heads, D), (ld, D, 1), 1)
        v.copy_(t)
        return v, buf

    def rest(v, buf):
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
        return buf[mask]

    def desc(x, dy, out):
        return _lib.HeadsDesc(X=x.data_ptr(), ldx=ld, hsx=D, w=w.data_ptr(), dY=dy.data_ptr(), lddy=ld,
                              hsdy=D, Y=out.data_ptr(), ldy=ld, hsy=D, heads=heads)

    stream = torch.cuda.current_stream().cuda_stream
    tail = (T, D, r, int(interleaved), 1e-6, 0, 1)
    v, buf = laid(x)
    assert d3.lib().dion3_qk_norm_rope(ctypes.byref(desc(v, v, v)), None, fr.data_ptr() or None,
                                       pos.data_ptr(), 64, *tail, stream) == 0
    assert torch.equal(v, y) and (rest(v, buf) == 7).all()
    size = ctypes.c_size_t()
    assert d3.lib().dion3_qk_norm_rope_grad_workspace_size(T, heads, 0, D, r, int(interleaved),
                                                           ctypes.byref(size)) == 0
    for over in (0, 1):
        (v, vb), (u, ub) = laid(x), laid(dy)
        out, ob = ((v, vb), (u, ub))[over]
        dw = torch.empty(2, D, device="cuda")
        ws = torch.full((size.value + 256,), 255, dtype=torch.uint8, device="cuda")
        at = ws.data_ptr() + (-ws.data_ptr()) % 256
        assert d3.lib().dion3_qk_norm_rope_grad(ctypes.byref(desc(v, u, out)), None, fr.data_ptr() or None,
                                                pos.data_ptr(), 64, dw.data_ptr(), *tail, at,
                                                size.value, stream) == 0
        assert torch.equal(out, want) and (rest(out, ob) == 7).all()
        assert torch.equal(dw[0], wdw) and not dw[1].any()


def test_refusals():
    q, k = torch.ones(4, 3, 64, dtype=BF, device="cuda"), torch.ones(4, 2, 64, dtype=BF, device="cuda")
    w, pos, fr = torch.ones(64, device="cuda"), torch.arange(4, device="cuda"), freqs_of(64).cuda()

    def bad(error, q=q, k=k, wq=w, wk=w, pos=pos, fr=fr, **kw):
        with pytest.raises(error):
            d3.qk_norm_rope(q, k, wq, wk, pos, fr, **kw)

    bad(TypeError, q=q.float())
    bad(TypeError, k=k.half())
    bad(TypeError, wq=w.half())
    bad(TypeError, wq=w.to(BF))                          # two types of weights
    bad(TypeError, fr=fr.float())
    bad(TypeError, pos=pos.float())
    bad(TypeError, pos=pos.cpu())
    bad(ValueError, k=None)
    bad(ValueError, k=k[:3])
    bad(ValueError, k=k[..., :32].contiguous())
    bad(ValueError, wq=w[:32])
    bad(ValueError, fr=freqs_of(66).cuda())
    bad(ValueError, q=q.transpose(1, 2), k=None, wk=None)
    bad(ValueError, q=q[:, :1].expand(4, 3, 64))
    bad(ValueError, q=torch.ones(2, 3, 2, 64, dtype=BF, device="cuda").transpose(0, 1), k=None, wk=None,
        pos=torch.zeros(3, 2, dtype=torch.int64, device="cuda"))
    bad((ValueError, RuntimeError), pos=pos[:3])
    bad(d3.Dion3Error, eps=-1.0)
    big = torch.ones(1, 1, 1032, dtype=BF, device="cuda")
    bad(d3.Dion3Error, q=big, k=None, wq=torch.ones(1032, device="cuda"), wk=None, pos=pos[:1])
