"""The layer operators at the ends of their ranges: activations of the largest
finite values, outputs in place of inputs, more elements than a launch's side
holds."""
import ctypes

import pytest
import torch

import orthogonalizing_optimizer_amd as d3

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_of_large_values(act, dtype):
    """From |z| = 128 on every activation is z or 0 and its slope 1 or 0, to
    the last bit (exp(-128) is below fp32's range), up to the type's largest
    finite value, where z^2 and z^3 leave fp32's."""
    top = torch.finfo(dtype).max
    z = [v for v in (128.0, 200.0, 1e3, 6e4, top / 2, top) if v <= top]
    if dtype == BF:
        z += [1e6, 1e12, 1.2e13, 2e13, 1e16, 1.8e19, 2e19, 1e30, 1e38]
    z = torch.tensor(z, dtype=dtype)
    z = torch.cat([z, -z]).cuda()[:, None].contiguous()
    on = (z > 0).to(dtype)
    # T x 1 by a weight of one: z itself, exactly
    y, pre = d3.linear(z, torch.ones(1, 1, dtype=dtype, device="cuda"), act=act, return_preact=True)
    assert torch.equal(pre, z) and torch.equal(y, torch.where(z > 0, z, torch.zeros_like(z)))
    dy = torch.full_like(z, 0.75)
    for zs in (z, d3.pack_f8(z)):
        dz, db = d3.act_grad(dy, zs, act, bias=True)
        assert torch.equal(dz, 0.75 * on), (act, dz)
        assert float(db) == 0.75 * float(on.float().sum())


@pytest.mark.parametrize("m", [40, 4096, 40000])
def test_norm_at_the_ends_of_its_sums(m):
    """Sums of squares past fp32's range give rstd = 0, below it none."""
    x = torch.ones(3, m, dtype=BF, device="cuda")
    x[0, 5], x[1] = 1.9e19, 1e-24
    y, _, rstd, _ = d3.add_rms_norm(x, torch.ones(m, device="cuda"), eps=1e-6)
    assert float(rstd[0]) == 0 and not y[0].any()
    assert abs(float(rstd[1]) - 1e3) <= 1e3 * 2.0 ** -22 and (y[2] == 1).all()


def room(nbytes):
    """Skip unless the GPU has this much free memory (and hand back torch's own)."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip("not enough free GPU memory")


def test_more_elements_than_a_grid_side_holds():
    """2^35 elements are 2^32 threads of 8: packing, its values and a gradient
    over no tokens past that, to the last row."""
    T, m = 1 << 24, 2080
    room(130 << 30)
    edge = (1 << 35) // m                              # the row of element 2^35
    rows = [0, 1, edge - 1, edge, edge + 1, T - 2, T - 1]
    g = torch.Generator().manual_seed(1)
    some = torch.randint(1, 5, (len(rows), m), generator=g).to(BF).cuda()
    x = torch.zeros(T, m, dtype=BF, device="cuda")
    x[rows] = some
    p = d3.pack_f8(x)
    del x                                              # (its values come back into its memory)
    part = d3.pack_f8(some)
    assert torch.equal(p.q[rows].view(torch.uint8), part.q.view(torch.uint8))
    assert torch.equal(p.scale[rows], part.scale)
    y = d3.unpack_f8(p, BF)
    assert torch.equal(y[rows], some)
    for t, width in ((p.q.view(torch.int64), m // 8), (y.view(torch.int64), m // 4)):
        assert t.shape == (T, width)
        full = sum(int((c != 0).any(1).sum()) for c in t.split(1 << 21))
        assert full == len(rows)                       # every other row was written as zeros
    del p, y, t
    n, m = 1 << 20, 32776                              # fp32: 2^35 elements and a little more
    room(150 << 30)
    G = torch.ones(n, m, device="cuda")
    none = torch.empty(0, n, dtype=BF, device="cuda"), torch.empty(0, m, dtype=BF, device="cuda")
    d3.linear_grad_weight(*none, out=G)
    assert not any(bool(c.any()) for c in G.split(1 << 17))
    del G
    torch.cuda.empty_cache()


# ------------------------------------------------------- outputs in place

def call(name, *args, size=None):
    """A C call on torch's current stream; size: its workspace call's arguments."""
    lib = d3.lib()
    tail = []
    if size is not None:
        nb = ctypes.c_size_t()
        assert getattr(lib, name + "_workspace_size")(*size, ctypes.byref(nb)) == 0
        ws = torch.empty(nb.value + 256, dtype=torch.uint8, device="cuda")
        tail = [ws.data_ptr() + (-ws.data_ptr()) % 256, nb.value]
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    assert getattr(lib, name)(*args, *tail, torch.cuda.current_stream().cuda_stream) == 0


def normal(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


CODE = {BF: 1, FP: 2}
ROWS = [(5, 1), (3, 20), (70, 515), (2600, 96), (1700, 2049), (900, 8200), (3, 16390), (600, 33003)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,m", ROWS)
def test_norm_writes_h_over_its_inputs(T, m, dtype):
    g = torch.Generator().manual_seed(T + m)
    x, r = normal(g, T, m, dtype=dtype), normal(g, T, m, dtype=dtype)
    w = 1 + normal(g, m, std=0.1, dtype=torch.float32)
    y, h, rstd, p = d3.add_rms_norm(x, w, residual=r, eps=1e-5, pack=True)
    for over in (0, 1):
        a = [x.clone(), r.clone()]
        Y, q, s = torch.empty_like(y), torch.empty_like(p.q), torch.empty_like(p.scale)
        rs = torch.empty_like(rstd)
        call("dion3_add_rms_norm", a[0], m, a[1], m, w, 0, a[over], m, Y, m, q, s, rs, T, m, 1e-5,
             CODE[dtype])
        assert torch.equal(a[over], h) and torch.equal(a[1 - over], (x, r)[1 - over])
        assert torch.equal(Y, y) and torch.equal(rs, rstd) and torch.equal(s, p.scale)
        assert torch.equal(q.view(torch.uint8), p.q.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,m", ROWS)
def test_norm_gradient_over_its_inputs(T, m, dtype):
    g = torch.Generator().manual_seed(T + m)
    h, dy, dh = (normal(g, T, m, dtype=dtype) for _ in range(3))
    w = 1 + normal(g, m, std=0.1, dtype=torch.float32)
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = d3.add_rms_norm_grad(dy, h, rstd, w, dh=dh)
    for over in (0, 1):
        a = [dy.clone(), dh.clone()]
        DW = torch.empty_like(dw)
        call("dion3_add_rms_norm_grad", a[0], m, h, m, rstd, w, 0, a[1], m, a[over], m, DW, T, m,
             CODE[dtype], size=(T, m))
        assert torch.equal(a[over], dx) and torch.equal(a[1 - over], (dy, dh)[1 - over])
        assert torch.equal(DW, dw)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,n", [(5, 1), (3, 20), (70, 515), (2600, 96), (1700, 2049), (300, 8200)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_act_gradient_over_its_inputs(act, T, n, dtype):
    g = torch.Generator().manual_seed(T + n)
    dy, z = normal(g, T, n, dtype=dtype), normal(g, T, n, std=2.0, dtype=dtype)
    dz, db = d3.act_grad(dy, z, act, bias=True)
    for over in (0, 1):
        a = [dy.clone(), z.clone()]
        DB = torch.empty_like(db)
        call("dion3_act_grad", a[0], n, a[1], n, None, None, a[over], n, DB, T, n,
             d3.ACTIVATIONS[act], CODE[dtype], size=(T, n))
        assert torch.equal(a[over], dz) and torch.equal(a[1 - over], (dy, z)[1 - over])
        assert torch.equal(DB, db)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,n,m", [(1, 20, 40), (1, 4099, 515), (9, 100, 64), (16, 520, 264),
                                   (70, 515, 77), (300, 260, 2100), (2100, 4101, 72),
                                   (2100, 72, 4100), (4100, 2120, 40)])
def test_products_over_their_addends(T, n, m, dtype):
    """Y is R, dX is R: few tokens, odd ends, split K, outputs in two rectangles."""
    g = torch.Generator().manual_seed(T + n + m)
    x, w, dz = normal(g, T, m, dtype=dtype), normal(g, n, m, dtype=dtype), normal(g, T, n, dtype=dtype)
    r, rx = normal(g, T, n, dtype=dtype), normal(g, T, m, dtype=dtype)
    y, z = d3.linear(x, w, act="silu", residual=r, return_preact=True)
    dx = d3.linear_grad_input(dz, w, residual=rx)
    Z = torch.empty_like(z)
    call("dion3_linear", x, m, w, m, None, 0, r, n, r, n, Z, n, T, n, m, d3.ACTIVATIONS["silu"],
         CODE[dtype], size=(x.data_ptr(), m, w.data_ptr(), m, T, n, m))
    assert torch.equal(r, y) and torch.equal(Z, z)
    call("dion3_linear_grad_input", dz, n, w, m, rx, m, rx, m, T, n, m, CODE[dtype],
         size=(dz.data_ptr(), n, w.data_ptr(), m, T, n, m))
    assert torch.equal(rx, dx)
