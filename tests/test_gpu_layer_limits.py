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
