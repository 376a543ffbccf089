"""The global gradient norm and clipping against the formula in 64 bits: many
tensors of mixed types, shapes and layouts, values at the ends of the types'
ranges, sums into other buffers, captures.

Bounds: squares are summed and gradients scaled in 64 bits, so the norm is off
by its own rounding to fp32, and a result by its rounding to fp32 and to its
type (2^-24 and half a step; 1.0001 is for the 64-bit parts)."""
import math

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, TINY, U, close, d

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
SHAPES = [(128, 512), (), (1,), (7,), (0, 5), (33, 515), (4096,), (3, 5, 7), (8191,), (8193,),
          (2, 70001), (300, 1)]


def rnd(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def placed(t, how):
    """t on the GPU in a layout of its own, sevens around it: (tensor, buffer)."""
    n = t.numel()
    if how == "transposed" and t.dim() == 2:
        buf = torch.full((n + 64,), 7, dtype=t.dtype, device="cuda")
        v = buf[:n].view(t.shape[1], t.shape[0]).t()
    elif how == "rows" and t.dim() == 2:
        ld = t.shape[1] + 5
        buf = torch.full((t.shape[0] * ld + 64,), 7, dtype=t.dtype, device="cuda")
        v = buf.as_strided(t.shape, (ld, 1), 3)
    else:
        off = 1 if how != "plain" else 0
        buf = torch.full((n + off + 64,), 7, dtype=t.dtype, device="cuda")
        v = buf[off:off + n].view(t.shape)
    v.copy_(t)
    return v, buf


def around(v, buf):
    """The buffer without v's elements."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
    return buf[mask]


def f32(x):
    """The library's max_norm is a float."""
    return float(torch.tensor(x, dtype=F32))


def norm64(ts, scale=1.0):
    return scale * math.sqrt(sum(float(d(t).square().sum()) for t in ts))


@pytest.mark.parametrize("how", ["plain", "off", "transposed", "rows"])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -12])
@pytest.mark.parametrize("ratio", [0.3, 1.5])
def test_norm_and_clip_in_place(ratio, scale, how):
    g = torch.Generator().manual_seed(1)
    host = [rnd(g, s, t, 0.1) for s in SHAPES for t in (F32, BF, FP)]
    put = [placed(t, how) for t in host]
    grads = [v for v, _ in put]
    want = norm64(host, scale)
    norm, norms = d3.grad_norm(grads, scale, per_tensor=True)
    assert norm.dtype == F32 and norm.dim() == 0 and norms.shape == (len(host),)
    assert abs(float(norm) - want) <= want * EPS32 * 1.001
    for t, n in zip(host, norms):
        one = norm64([t], scale)
        assert abs(float(n) - one) <= one * EPS32 * 1.001
    most = f32(ratio * want)
    got = d3.clip_grad_norm(grads, most, scale)
    assert torch.equal(got, norm)
    c = scale * min(1.0, most / want)
    for t, (v, buf) in zip(host, put):
        w = d(t) * c
        close(v, w, w.abs() * (U[t.dtype] + (0 if t.dtype == F32 else 1.01 * EPS32)) * 1.0001 + TINY[t.dtype], (t.shape, t.dtype))
        if c == 1.0:
            assert torch.equal(v.cpu(), t)
        assert (around(v, buf) == 7).all()


@pytest.mark.parametrize("how_m", ["plain", "off", "rows"])
@pytest.mark.parametrize("how", ["plain", "transposed", "rows"])
@pytest.mark.parametrize("ratio", [0.3, 1.5])
def test_clip_into_sums(ratio, how, how_m):
    g = torch.Generator().manual_seed(2)
    host = [rnd(g, s, t, 0.1) for s in SHAPES for t in (F32, BF, FP)]
    if how == "transposed" and how_m == "rows":
        host = [t for t in host if t.dim() != 2]          # no common layout: refused below
    sums = [rnd(g, t.shape, F32) for t in host]
    grads = [placed(t, how)[0] for t in host]
    if how == "transposed":
        put = [placed(t, "transposed") for t in sums]     # equal strides
    else:
        put = [placed(t, how_m) for t in sums]
    want = norm64(host)
    most = f32(ratio * want)
    norm = d3.clip_grad_norm(grads, most, into=[v for v, _ in put])
    assert abs(float(norm) - want) <= want * EPS32 * 1.001
    c = min(1.0, most / want)
    for t, v, m, (out, buf) in zip(host, grads, sums, put):
        assert torch.equal(v.cpu(), t)
        w = d(m) + c * d(t)
        close(out, w, w.abs() * EPS32 * 1.0001 + 1e-45, t.shape)
        assert (around(out, buf) == 7).all()


def test_more_tensors_than_a_launch_holds():
    g = torch.Generator().manual_seed(3)
    sizes = [1 + (37 * i) % 900 for i in range(700)]
    sizes[100:160] = [0] * 60
    host = [rnd(g, (n,), (F32, BF, FP)[i % 3]) for i, n in enumerate(sizes)]
    grads = [t.cuda() for t in host]
    grads[5] = None
    host[5] = torch.zeros(3)
    norm, norms = d3.grad_norm(grads, per_tensor=True)
    want = norm64(host)
    assert abs(float(norm) - want) <= want * EPS32 * 1.001
    for t, n in zip(host, norms.tolist()):
        assert abs(n - norm64([t])) <= norm64([t]) * EPS32 * 1.001
    d3.clip_grad_norm(grads, f32(want / 4))
    for t, v in zip(host, grads):
        if v is not None:
            w = d(t) * f32(want / 4) / want
            close(v, w, w.abs() * (U[t.dtype] + (0 if t.dtype == F32 else 1.01 * EPS32)) * 1.0001 + TINY[t.dtype])


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_ends_of_the_range(dtype):
    """Squares of the type's largest and smallest values stay in the sum."""
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).tiny / 4
    a = torch.tensor([top, -top, 1.0], dtype=dtype, device="cuda")
    want = math.sqrt(2.0) * float(torch.tensor(top, dtype=dtype))
    norm = d3.grad_norm([a], scale=2.0 ** -1)
    assert abs(float(norm) - want / 2) <= want * EPS32
    b = torch.tensor([low, low, low, -low], dtype=dtype, device="cuda")
    assert float(d3.grad_norm([b])) == 2 * float(b[0])
    norm = d3.clip_grad_norm([a], 1.0, scale=2.0 ** -1)
    w = torch.tensor([math.sqrt(0.5), -math.sqrt(0.5), 1 / want], dtype=torch.float64)
    close(a, w, w.abs() * (U[dtype] + (0 if dtype == F32 else 1.01 * EPS32)) * 1.0001 + TINY[dtype])


def test_nan_infinity_and_bounds():
    def lists():
        return [torch.tensor([1.0, -2.0], device="cuda"), torch.tensor([4.0, 3.0], device="cuda")]
    a = lists()
    a[1][0] = math.inf
    assert math.isinf(float(d3.clip_grad_norm(a, 1.0)))
    assert a[0].tolist() == [0.0, 0.0] and math.isnan(float(a[1][0])) and float(a[1][1]) == 0
    a = lists()
    a[1][0] = math.nan
    assert math.isnan(float(d3.clip_grad_norm(a, 1.0)))
    assert all(bool(torch.isnan(t).all()) for t in a)
    a = lists()
    assert float(d3.clip_grad_norm(a, math.inf)) == float(d3.grad_norm(lists()))
    assert torch.equal(torch.cat(a), torch.cat(lists()))
    d3.clip_grad_norm(a, 0.0)
    assert not torch.cat(a).any()
    assert float(d3.clip_grad_norm(a, 0.0)) == 0 and not torch.cat(a).any()   # 0 / 0 is no clipping


def test_no_gradients():
    assert float(d3.grad_norm([])) == 0 and float(d3.clip_grad_norm([None, None], 1.0)) == 0
    e = torch.empty(0, 3, device="cuda")
    norm, norms = d3.grad_norm([e, e], per_tensor=True)
    assert float(norm) == 0 and norms.tolist() == [0.0, 0.0]
    assert float(d3.clip_grad_norm([e, e], 1.0)) == 0


def test_more_than_2_31_elements():
    n = (1 << 31) + 4099
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough free GPU memory")
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[0], t[1 << 31], t[-1] = 1.0, 2.0, 2.0
    assert float(d3.grad_norm([t])) == 3.0
    assert float(d3.clip_grad_norm([t], 1.5)) == 3.0
    assert [float(t[i]) for i in (0, 1, 1 << 31, n - 1)] == [0.5, 0.0, 1.0, 1.0]
    assert float(d3.grad_norm([t])) == 1.5


def test_captured_and_on_another_stream():
    g = torch.Generator().manual_seed(4)
    host = [rnd(g, s, t) for s in SHAPES for t in (F32, BF)]
    static = [t.cuda() for t in host]
    sums = [torch.zeros(t.shape, device="cuda") for t in host]
    want = norm64(host)
    d3.clip_grad_norm([t.clone() for t in static], 1.0)            # warm
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        norm = d3.clip_grad_norm(static, 0.5 * want, into=sums)
    for k in range(4):
        for t, h in zip(static, host):
            t.copy_(h * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.zeros(t.shape, device="cuda") for t in host]
        n = d3.clip_grad_norm(static, 0.5 * want, into=eager)
        assert torch.equal(n, norm)
        for a, b in zip(sums, eager):
            assert torch.equal(a, b)
            a.zero_()
    with torch.cuda.stream(s):
        b = d3.grad_norm(static)
    s.synchronize()
    assert torch.equal(b, norm)


def test_refusals():
    a, b = torch.ones(4, 4, device="cuda"), torch.ones(4, 4, device="cuda")
    p = torch.nn.Parameter(a.clone())
    with pytest.raises(TypeError):
        d3.clip_grad_norm([p], 1.0)
    with pytest.raises(TypeError):
        d3.clip_grad_norm([a, a.double()], 1.0)
    with pytest.raises(TypeError):
        d3.clip_grad_norm([a, torch.ones(3)], 1.0)
    with pytest.raises(ValueError):
        d3.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(ValueError):
        d3.clip_grad_norm([a, b], 1.0, into=[a, a])
    for into in ([b, a], [a, torch.ones(4, 4, device="cuda")]):     # sums that are gradients
        with pytest.raises(ValueError):
            d3.clip_grad_norm([a, b], 1.0, into=into)
    with pytest.raises(ValueError):
        d3.clip_grad_norm([a], 1.0, into=[a, b])
    with pytest.raises(ValueError):
        d3.clip_grad_norm([a], 1.0, into=[torch.ones(4, 5, device="cuda")])
    with pytest.raises(TypeError):
        d3.clip_grad_norm([a], 1.0, into=[torch.ones(4, 4, device="cuda", dtype=BF)])
    with pytest.raises(TypeError):
        d3.clip_grad_norm([a, b], 1.0, into=[b, None])
    with pytest.raises(ValueError):
        d3.clip_grad_norm([a[:, ::2]], 1.0)
    with pytest.raises(ValueError):
        d3.clip_grad_norm([a[:1].expand(4, 4)], 1.0)
    with pytest.raises(ValueError):                       # no common layout
        d3.clip_grad_norm([torch.ones(5, 4, device="cuda").t()], 1.0,
                          into=[torch.zeros(4, 9, device="cuda")[:, :5]])
    for bad in (-1.0, math.nan):
        with pytest.raises(d3.Dion3Error):
            d3.clip_grad_norm([a], bad)
    for bad in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(d3.Dion3Error):
            d3.grad_norm([a], bad)
    assert (a == 1).all() and (b == 1).all()
    assert abs(float(d3.grad_norm([a, a])) - math.sqrt(32.0)) <= 6 * EPS32       # reads only


def test_optimizer_clips_its_gradients():
    g = torch.Generator().manual_seed(5)
    w = [rnd(g, s, F32, 0.02).cuda().requires_grad_(True) for s in ((128, 512), (64, 96))]
    v = [p.detach().clone().requires_grad_(True) for p in w]
    grads = [rnd(g, p.shape, F32).cuda() for p in w]
    a, b = d3.Dion3(w), d3.Dion3(v)
    for p, q, t in zip(w, v, grads):
        p.grad, q.grad = t.clone(), t.clone()
    norm = a.clip_grad_norm(1.0)
    want = norm64(grads)
    assert abs(float(norm) - want) <= want * EPS32 * 1.001
    d3.clip_grad_norm([q.grad for q in v], 1.0)
    a.step()
    b.step()
    for p, q in zip(w, v):
        assert torch.equal(p, q) and torch.equal(a.momentum(p), b.momentum(q))
    # 16-bit gradients summed into the momenta: no .grad needed
    h = [t.to(BF) for t in grads]
    before = [a.momentum(p).clone() for p in w]
    for p in w:
        p.grad = None
    d3.clip_grad_norm(h, 1.0, into=[a.accumulate_grad(p) for p in w])
    for p, m, t in zip(w, before, h):
        wm = d(m) + d(t) / norm64(h)
        close(a.momentum(p), wm, wm.abs() * EPS32 * 1.0001)
    with pytest.raises(RuntimeError):
        a.clip_grad_norm(1.0)
    a.step()
    a.clip_grad_norm(1.0)
