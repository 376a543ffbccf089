"""The layer operators at the ends of their ranges: activations of the largest
finite values, outputs in place of inputs, more elements than a launch's side
holds."""
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
