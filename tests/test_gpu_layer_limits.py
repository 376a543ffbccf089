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
    """A C call on torch's current stream; size: its workspace call's
    arguments.  The workspace is exactly as large as asked for, and what lies
    behind it stays as it was."""
    lib = d3.lib()
    tail, ws = [], None
    if size is not None:
        nb = ctypes.c_size_t()
        assert getattr(lib, name + "_workspace_size")(*size, ctypes.byref(nb)) == 0
        ws = torch.full((nb.value + 256 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        at = -ws.data_ptr() % 256
        tail = [ws.data_ptr() + at, nb.value]
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    assert getattr(lib, name)(*args, *tail, torch.cuda.current_stream().cuda_stream) == 0
    if ws is not None:
        assert (ws[:at] == 0xA5).all() and (ws[at + nb.value:] == 0xA5).all()


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


# ---------------------------------- what lies between and behind the outputs

class Out:
    """A [T, m] output at an odd place in a buffer of sevens."""

    def __init__(self, T, m, dtype, ld=None, off=0):
        self.ld = ld or m
        self.buf = torch.full((T * self.ld + off + 512,), 7, dtype=dtype, device="cuda")
        self.t = self.buf.as_strided((T, m), (self.ld, 1), off)
        self.ptr = self.t.data_ptr()

    def take(self):
        """Its values; all around them still sevens."""
        v = self.t.clone()
        self.t.fill_(7)
        assert (self.buf == 7).all()
        return v


@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1), (16, 8)])
@pytest.mark.parametrize("T,m", [(1, 1), (3, 20), (70, 515), (9, 2049), (3, 16390), (3, 33003)])
def test_row_operators_write_their_outputs_only(T, m, pad, off):
    g = torch.Generator().manual_seed(T * m + pad)
    x, r, dy = (normal(g, T, m) for _ in range(3))
    w = 1 + normal(g, m, std=0.1, dtype=torch.float32)
    y, h, rstd, p = d3.add_rms_norm(x, w, residual=r, pack=True)
    mp, ld = p.q.shape[1], m + pad
    Y, H = Out(T, m, BF, ld, off), Out(T, m, BF, ld, off)
    Q, S, RS = Out(T, mp, torch.uint8, off=16), Out(T, mp // 32, torch.uint8, off=off), Out(T, 1, torch.float32, off=off)
    call("dion3_add_rms_norm", x, m, r, m, w, 0, H.ptr, ld, Y.ptr, ld, Q.ptr, S.ptr, RS.ptr, T, m,
         1e-6, 1)
    assert torch.equal(Y.take(), y) and torch.equal(H.take(), h)
    assert torch.equal(Q.take(), p.q.view(torch.uint8)) and torch.equal(S.take(), p.scale)
    assert torch.equal(RS.take()[:, 0], rstd)
    call("dion3_pack_f8", y, m, Q.ptr, S.ptr, T, m, 1)
    assert torch.equal(Q.take(), p.q.view(torch.uint8)) and torch.equal(S.take(), p.scale)
    for t, code in ((BF, 1), (FP, 2), (torch.float32, 0)):
        V = Out(T, m, t, ld, off)
        call("dion3_unpack_f8", p.q, p.scale, V.ptr, ld, T, m, code)
        assert torch.equal(V.take(), d3.unpack_f8(p, t))
    dx, dw = d3.add_rms_norm_grad(dy, h, rstd, w, dh=r)
    DX, DW = Out(T, m, BF, ld, off), Out(1, m, torch.float32, off=off)
    call("dion3_add_rms_norm_grad", dy, m, h, m, rstd, w, 0, r, m, DX.ptr, ld, DW.ptr, T, m, 1,
         size=(T, m))
    assert torch.equal(DX.take(), dx) and torch.equal(DW.take()[0], dw)
    dz, db = d3.act_grad(dy, x, "silu", bias=True)
    call("dion3_act_grad", dy, m, x, m, None, None, DX.ptr, ld, DW.ptr, T, m, 4, 1, size=(T, m))
    assert torch.equal(DX.take(), dz) and torch.equal(DW.take()[0], db)


@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1), (16, 8)])
@pytest.mark.parametrize("T,n,m", [(1, 1, 1), (1, 4099, 515), (9, 100, 64), (16, 24, 520), (5, 7, 9),
                                   (70, 515, 77), (300, 260, 2100), (2100, 4101, 72),
                                   (4100, 2120, 40), (5000, 100, 60), (0, 33, 20)])
def test_products_write_their_outputs_only(T, n, m, pad, off):
    g = torch.Generator().manual_seed(T + n + m + pad)
    x, w, dz, r = normal(g, T, m), normal(g, n, m), normal(g, T, n), normal(g, T, n)
    y, z = d3.linear(x, w, act="silu", residual=r, return_preact=True)
    Y, Z = Out(T, n, BF, n + pad, off), Out(T, n, BF, n + pad, off)
    call("dion3_linear", x, m, w, m, None, 0, r, n, Y.ptr, n + pad, Z.ptr, n + pad, T, n, m, 4, 1,
         size=(x.data_ptr(), m, w.data_ptr(), m, T, n, m))
    assert torch.equal(Y.take(), y) and torch.equal(Z.take(), z)
    DX = Out(T, m, BF, m + pad, off)
    call("dion3_linear_grad_input", dz, n, w, m, None, 0, DX.ptr, m + pad, T, n, m, 1,
         size=(dz.data_ptr(), n, w.data_ptr(), m, T, n, m))
    assert torch.equal(DX.take(), d3.linear_grad_input(dz, w))
    p = d3.pack_f8(x)
    for a, s in ((x, None), (p.q, p.scale)):
        G = Out(n, m, torch.float32, m + pad, off)
        sp = None if s is None else s.data_ptr()
        call("dion3_linear_grad_weight", dz, n, a, m, sp, G.ptr, m + pad, 0, T, n, m, 1,
             size=(dz.data_ptr(), n, a.data_ptr(), m, sp, T, n, m))
        assert torch.equal(G.take(), d3.linear_grad_weight(dz, x if s is None else p))
