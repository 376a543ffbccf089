"""Weight gradients summed into the optimizer's momentum by the kernels: which
backward passes do so, in what order over streams, and around graphs."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def setting(seed, T=70, n=136, m=264):
    g = torch.Generator().manual_seed(seed)
    x, dy = rnd(g, T, m, dtype=BF).requires_grad_(True), rnd(g, T, n, dtype=BF)
    w = rnd(g, n, m, std=0.05).requires_grad_(True)
    return x, w, dy, d3.Dion3([w], lr=0.02, fraction=0.25)


@pytest.mark.parametrize("checkpoint", ["f8", "full"])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_passes_that_do_not_ask_for_the_weight(act, checkpoint):
    """Input gradients leave the momentum and the step alone; the weight's
    gradient as a value is the one that a whole pass sums."""
    x, w, dy, opt = setting(1)
    y = d3.linear_layer(x, w, act=act, checkpoint=checkpoint, into=opt)
    gx, = torch.autograd.grad(y, x, dy, retain_graph=True)
    y.backward(dy, inputs=[x], retain_graph=True)
    assert torch.equal(x.grad, gx)
    gw, = torch.autograd.grad(y, w, dy, retain_graph=True)
    assert not opt.momentum(w).any() and w.grad is None
    before = w.detach().clone()
    opt.step()
    assert torch.equal(w.detach(), before)
    y.backward(dy)
    assert torch.equal(opt.momentum(w), gw) and w.grad is None
    opt.step()
    assert not torch.equal(w.detach(), before)
