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


@pytest.mark.parametrize("shared", [True, False])
def test_two_backward_passes_on_two_streams(shared):
    """One weight on two streams: the sums and the momentum's first zeros do not
    meet.  Shared: two branches of one backward pass; else two passes."""
    T, n, m = 8192, 512, 1024
    batches = [setting(s, T, n, m)[::2] for s in (2, 3)]
    w0 = setting(2, T, n, m)[1].detach()
    want = None
    for streams in [[torch.cuda.current_stream()] * 2, [torch.cuda.Stream() for _ in range(2)]]:
        w = w0.clone().requires_grad_(True)
        opt = d3.Dion3([w], lr=0.02, fraction=0.25)
        torch.cuda.synchronize()
        ys = []
        for s, (x, _) in zip(streams, batches):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                ys.append(d3.linear_layer(x, w, into=opt))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        if shared:
            torch.autograd.backward(ys, [dy for _, dy in batches])
        else:
            for s, y, (_, dy) in zip(streams, ys, batches):
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    y.backward(dy)
        opt.step()
        got = [opt.momentum(w).clone(), w.detach().clone()]
        if want is None:
            want = got
        # (two sums into zeros: a + b is b + a, whichever came first)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_sum_behind_a_step_on_another_stream():
    """A backward pass of an older forward pass, on its own stream, after a
    step on another: the sum follows the step."""
    T, n, m = 4096, 512, 1024
    x, w, dy, opt = setting(4, T, n, m)
    x2, _, dy2, _ = setting(5, T, n, m)
    w0 = w.detach().clone()
    results = []
    for side in (torch.cuda.current_stream(), torch.cuda.Stream()):
        v = w0.clone().requires_grad_(True)
        opt = d3.Dion3([v], lr=0.02, fraction=0.25)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ys = [d3.linear_layer(t, v, into=opt) for t in (x, x2)]
        torch.cuda.current_stream().wait_stream(side)
        ys[0].backward(dy)
        opt.step()
        with torch.cuda.stream(side):
            ys[1].backward(dy2)
        results.append(opt.momentum(v).clone())          # (the current stream waits for the sum)
    assert torch.equal(*results)


def test_steps_around_a_captured_backward_pass():
    """Capturing steps nothing; a replay announced by accumulate_grad is stepped
    as the eager pass is."""
    batches = [setting(s)[::2] for s in (6, 7, 8, 9)]
    w0 = setting(6)[1].detach()

    def fresh():
        w = w0.clone().requires_grad_(True)
        return w, d3.Dion3([w], lr=0.02, fraction=0.25)

    w, opt = fresh()
    want = []
    for x, dy in batches:
        d3.linear_layer(x.detach(), w, act="silu", into=opt).backward(dy)
        opt.step()
        want.append([w.detach().clone(), opt.momentum(w).clone()])
    w, opt = fresh()
    x, dy = (t.detach().clone() for t in batches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                     # first launches
        v, other = fresh()
        d3.linear_layer(x, v, act="silu", into=other).backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    opt.momentum(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d3.linear_layer(x, w, act="silu", into=opt).backward(dy)
    opt.step()
    assert torch.equal(w.detach(), w0) and not opt.momentum(w).any()
    for (xb, dyb), (ww, mw) in zip(batches, want):
        x.copy_(xb.detach())
        dy.copy_(dyb)
        opt.accumulate_grad(w)
        graph.replay()
        opt.step()
        torch.cuda.synchronize()
        assert torch.equal(w.detach(), ww) and torch.equal(opt.momentum(w), mw)


@pytest.mark.parametrize("lead", [(0,), (2, 0)])
def test_no_tokens(lead):
    """A batch without tokens: zero gradients, nothing added to the momentum."""
    x, w, _, opt = setting(10)
    x = x.detach()[:0].view(*lead, 264).requires_grad_(True)
    b = torch.zeros(136, device="cuda", requires_grad=True)
    n1 = torch.ones(264, device="cuda", requires_grad=True)
    for into in (None, opt):
        y, h, packed = d3.rms_norm_residual(x, n1, residual=x, pack=True)
        out = d3.linear_layer(y, w, b, act="silu", checkpoint=packed, into=into)
        assert out.shape == (*lead, 136)
        out.sum().backward()
        assert x.grad.shape == x.shape and not b.grad.any() and not n1.grad.any()
    assert not w.grad.any() and not opt.momentum(w).any()
