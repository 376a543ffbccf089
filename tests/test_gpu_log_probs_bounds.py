"""Log probabilities where a term of no weight is far from the rest: the product
of its zero and its distance has to stay zero."""
import math

import numpy as np
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import TINY, U, close
from tests.test_gpu_log_probs_far import Far, check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_parts_far_apart():
    """Sums whose residual is large, beside a logit that dwarfs them."""
    scale = np.float32(0.7)
    x = -5e8 - 32.0 * np.arange(4096)
    z = x * float(scale)
    r = z - z.astype(np.float32).astype(np.float64)
    v = float(x[np.argmax(r)])
    assert r.max() > 12 and np.float32(v) == v
    t = torch.full((2, 60000), v)
    t[0, 59999], t[1, 0] = 1e31, 1e31
    check(t, torch.tensor([59999, 0]), float(scale))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gh", [1e6, 1e12])
def test_large_gradient_of_the_entropy(gh, dtype):
    """Columns without a probability get no gradient, however large it is."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 300, generator=g)
    x[:, 250:] = -math.inf
    x[1, 200:250] = -2000.0
    x = x.to(dtype)
    t = torch.tensor([1, 2, 3])
    _, stats, H, _, _ = d3.log_probs(x.cuda(), t.cuda(), entropy=True)
    gl, big = torch.ones(3), torch.full((3,), gh)
    dx = d3.log_probs_grad(gl.cuda(), x.cuda(), t.cuda(), stats, entropy=H, dentropy=big.cuda())
    want, off = Far(x, t, 1.0).grad(gl, big)
    close(dx, want, (want.abs() + off) * U[dtype] + off + TINY[dtype])
    assert not dx[:, 250:].any() and not dx[1, 200:].any()
