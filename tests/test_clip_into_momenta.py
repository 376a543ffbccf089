"""Clipped gradients summed into an optimizer's momenta: which parameters the
next step counts.  On the CPU the refusals and the bookkeeping, with the
clipping's call replaced by its formula; on the GPU the whole of it."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from orthogonalizing_optimizer_amd import clip, optim
from tests.layer_ref import EPS32, close, d


def formula(grads, max_norm, scale=1.0, into=None, ws=None):
    have = [(g, m) for g, m in zip(grads, into) if g is not None]
    norm = scale * sum(float(g.double().square().sum()) for g, _ in have) ** 0.5
    c = 1.0 if norm <= max_norm else max_norm / norm
    for g, m in have:
        m.add_(g.float(), alpha=c * scale)
    return torch.tensor(norm)


def setting(device="cpu"):
    g = torch.Generator().manual_seed(3)
    ps = [torch.randn(s, generator=g).to(device).requires_grad_(True) for s in ((8, 12), (6, 6), (4, 20))]
    grads = [torch.randn(p.shape, generator=g).to(device) for p in ps]
    return ps, grads, d3.Dion3(ps)


def test_names_the_parameters_with_a_gradient(monkeypatch):
    monkeypatch.setattr(clip, "clip_grad_norm", formula)
    ps, grads, opt = setting()
    norm = opt.accumulate_clipped(ps, [grads[0], None, grads[2]], 1.0)
    want = (d(grads[0]).square().sum() + d(grads[2]).square().sum()).sqrt()
    assert abs(float(norm) - float(want)) <= 1e-6 * float(want)
    assert opt._accumulated == {ps[0], ps[2]} and "momentum" not in opt.state.get(ps[1], ())
    for i in (0, 2):
        assert torch.allclose(opt.momentum(ps[i]), grads[i] / want.float(), atol=1e-6)
    opt.accumulate_clipped(ps[1:2], grads[1:2], 1.0)
    assert opt._accumulated == set(ps)


def test_no_gradients_at_all():
    ps, _, opt = setting()
    before = [p.detach().clone() for p in ps]
    assert float(opt.accumulate_clipped(ps, [None] * 3, 1.0)) == 0
    opt.step()                                        # (steps nothing: there is no GPU here)
    assert all(torch.equal(p, b) for p, b in zip(ps, before)) and not opt._accumulated


def test_refused_calls_name_nothing(monkeypatch):
    ps, grads, opt = setting()
    other = torch.randn(3, 3, requires_grad=True)
    for error, args in ((TypeError, (ps, grads, 1.0)),                        # (not on a GPU)
                        (ValueError, (ps, grads[:2], 1.0)),
                        (ValueError, ([other], [torch.ones(3, 3)], 1.0)),
                        (ValueError, ([ps[0], ps[0]], [grads[0], grads[0]], 1.0))):
        with pytest.raises(error):
            opt.accumulate_clipped(*args)
        assert not opt._accumulated
    opt.clip_grad_norm(1.0)                           # (refused while any is named)


def test_order_of_streams_and_captures(monkeypatch):
    monkeypatch.setattr(clip, "clip_grad_norm", formula)
    monkeypatch.setattr(optim, "_stream", lambda t: "b")
    waits, captured = [], set()
    monkeypatch.setattr(optim, "_follow", lambda here, last: waits.append((here, last)))
    monkeypatch.setattr(optim, "_hold", lambda t, stream: None)
    monkeypatch.setattr(optim, "_capturing", lambda s: s in captured)
    ps, grads, opt = setting()
    for p in ps:
        opt.momentum(p)
        opt._last[p] = "a"
    opt.accumulate_clipped(ps[:2], [grads[0], None], 1.0)
    assert waits == [("b", "a")] and opt._accumulated == {ps[0]}
    captured.add("b")
    opt.accumulate_clipped(ps[1:], grads[1:], 1.0)    # part of a capture: named by nobody
    assert opt._accumulated == {ps[0]}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parameter_without_a_gradient_stays(dtype):
    ps, grads, opt = setting("cuda")
    for p, g in zip(ps, grads):                       # a step, so that momenta hold something
        p.grad = g.clone()
    opt.step()
    for p in ps:
        p.grad = None
    before = [(p.detach().clone(), opt.momentum(p).clone()) for p in ps]
    h = [g.to(dtype) for g in grads]
    norm = opt.accumulate_clipped(ps, [h[0], None, h[2]], 1.0, scale=0.5)
    want = 0.5 * float((d(h[0]).square().sum() + d(h[2]).square().sum()).sqrt())
    assert abs(float(norm) - want) <= want * EPS32 * 1.001
    for i in (0, 2):
        wm = d(before[i][1]) + 0.5 * d(h[i]) / want
        close(opt.momentum(ps[i]), wm, wm.abs() * EPS32 * 1.0001)
    opt.step()
    assert torch.equal(ps[1], before[1][0]) and torch.equal(opt.momentum(ps[1]), before[1][1])
    assert not torch.equal(ps[0], before[0][0]) and not torch.equal(ps[2], before[2][0])


@pytest.mark.gpu
def test_refused_call_leaves_the_parameters():
    ps, grads, opt = setting("cuda")
    before = [p.detach().clone() for p in ps]
    with pytest.raises(ValueError):
        opt.accumulate_clipped(ps, [grads[0], None, grads[1]], 1.0)      # another shape
    with pytest.raises(d3.Dion3Error):
        opt.accumulate_clipped(ps, grads, -1.0)
    opt.step()
    assert all(torch.equal(p, b) for p, b in zip(ps, before))
    assert not any(opt.momentum(p).any() for p in ps)


@pytest.mark.gpu
def test_captured_and_replayed():
    ps, grads, opt = setting("cuda")
    ps.append(torch.randn(5, 7, device="cuda").requires_grad_(True))    # never a gradient, no momentum
    opt.add_param_group({"params": [ps[3]]})
    grads.append(None)
    for p in ps[:3]:
        opt.momentum(p)
    opt.accumulate_clipped(ps, [grads[0], None, grads[2], None], 1.0)
    opt.step()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        norm = opt.accumulate_clipped(ps, [grads[0], None, grads[2], None], 1.0)
    assert not opt._accumulated
    for k in range(4):
        for i in (0, 2):
            grads[i].mul_(1.0 + k)
            opt.accumulate_grad(ps[i])
        before = [(p.detach().clone(), opt.momentum(p).clone()) for p in ps[:3]]
        graph.replay()
        torch.cuda.synchronize()
        want = float((d(grads[0]).square().sum() + d(grads[2]).square().sum()).sqrt())
        assert abs(float(norm) - want) <= want * EPS32 * 1.001
        for i in (0, 2):
            wm = d(before[i][1]) + d(grads[i]) * min(1.0, 1.0 / want)
            close(opt.momentum(ps[i]), wm, wm.abs() * EPS32 * 1.0001)
        opt.step()
        assert torch.equal(ps[1], before[1][0]) and torch.equal(opt.momentum(ps[1]), before[1][1])
        assert not torch.equal(ps[0], before[0][0])
    assert "momentum" not in opt.state.get(ps[3], ())
