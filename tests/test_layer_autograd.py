"""The autograd side of the layer operators, on the CPU: which gradients a
backward pass asks for, and what the optimizer's momentum receives.  The
kernels are replaced by their formulas; what runs here is the package's own
bookkeeping."""
import copy

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from orthogonalizing_optimizer_amd import layer, optim


@pytest.fixture(autouse=True)
def formulas(monkeypatch):
    """The calls of the library that linear_layer(..., checkpoint="full") makes."""
    def linear(x, w, bias=None, act="none", residual=None, return_preact=False):
        z = x @ w.t() if bias is None else x @ w.t() + bias
        return (z if residual is None else z + residual), (z if return_preact else None)

    def grad_weight(dz, x, out=None, accumulate=False):
        dw = dz.reshape(-1, dz.shape[-1]).t() @ x.reshape(-1, x.shape[-1])
        if out is None:
            return dw
        return out.add_(dw) if accumulate else out.copy_(dw)

    monkeypatch.setattr(layer, "linear", linear)
    monkeypatch.setattr(layer, "act_grad",
                        lambda dy, z, act, bias=False: (dy, dy.sum(0) if bias else None))
    monkeypatch.setattr(layer, "linear_grad_input", lambda dz, w: dz @ w)
    monkeypatch.setattr(layer, "linear_grad_weight", grad_weight)


def setting(seed=1, T=6, n=4, m=5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, m, generator=g, requires_grad=True)
    w = torch.randn(n, m, generator=g, requires_grad=True)
    b = torch.randn(n, generator=g, requires_grad=True)
    dy = torch.randn(T, n, generator=g)
    opt = d3.Dion3([w])
    y = d3.linear_layer(x, w, b, checkpoint="full", into=opt)
    return x, w, b, dy, opt, y


def untouched(opt, w):
    return not opt._accumulated and not opt.momentum(w).any() and w.grad is None


def test_whole_backward_pass_sums_into_the_momentum():
    x, w, b, dy, opt, y = setting()
    y.backward(dy)
    assert torch.equal(opt.momentum(w), dy.t() @ x.detach()) and w.grad is None
    assert w in opt._accumulated
    assert torch.equal(x.grad, dy @ w.detach()) and torch.equal(b.grad, dy.sum(0))


def test_pass_for_other_inputs_leaves_the_momentum():
    x, w, b, dy, opt, y = setting()
    gx, gb = torch.autograd.grad(y, (x, b), dy, retain_graph=True)
    assert torch.equal(gx, dy @ w.detach()) and torch.equal(gb, dy.sum(0))
    assert untouched(opt, w)
    y.backward(dy, inputs=[x], retain_graph=True)
    assert torch.equal(x.grad, gx) and b.grad is None
    assert untouched(opt, w)
    y.backward(dy, inputs=[b, w])              # asked for by name
    assert torch.equal(opt.momentum(w), dy.t() @ x.detach()) and w in opt._accumulated


def test_weight_gradient_as_a_value():
    x, w, b, dy, opt, y = setting()
    gw, = torch.autograd.grad(y, w, dy, retain_graph=True)
    assert torch.equal(gw, dy.t() @ x.detach())
    gw, gx = torch.autograd.grad(y, (w, x), dy)
    assert torch.equal(gw, dy.t() @ x.detach()) and torch.equal(gx, dy @ w.detach())
    assert untouched(opt, w)


def test_weight_used_twice():
    x, w, _, _, opt, _ = setting(n=5)
    y1 = d3.linear_layer(x, w, checkpoint="full", into=opt)
    y = d3.linear_layer(y1, w, checkpoint="full", into=opt)
    dy = torch.randn_like(y)
    torch.autograd.grad(y, x, dy, retain_graph=True)
    torch.autograd.grad(y, y1, dy, retain_graph=True)
    assert untouched(opt, w)
    with torch.no_grad():
        want = dy.t() @ y1 + (dy @ w).t() @ x
    gw, = torch.autograd.grad(y, w, dy, retain_graph=True)
    assert torch.allclose(gw, want, rtol=1e-5, atol=1e-5) and untouched(opt, w)
    y.backward(dy)
    assert torch.allclose(opt.momentum(w), want, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_layer(reentrant):
    from torch.utils.checkpoint import checkpoint
    x, w, _, dy, opt, _ = setting()
    y = checkpoint(lambda t: d3.linear_layer(t, w, checkpoint="full", into=opt), x,
                   use_reentrant=reentrant)
    y.backward(dy)
    assert torch.equal(opt.momentum(w), dy.t() @ x.detach())
    assert torch.equal(x.grad, dy @ w.detach())


# ---------------------------------------------------- the order of the sums

class Streams:
    """Streams as names: the current one, those being captured, and the waits asked for."""

    def __init__(self, monkeypatch):
        self.here, self.captured, self.waits = "a", set(), []
        monkeypatch.setattr(optim, "_stream", lambda t: self.here)
        monkeypatch.setattr(optim, "_capturing", lambda s: s in self.captured)
        self.held = []
        monkeypatch.setattr(optim, "_follow", lambda here, last: self.waits.append((here, last)))
        monkeypatch.setattr(optim, "_hold", lambda t, stream: self.held.append((t, stream)))

    def sums(self, opt, w, here):
        """The waits before a gradient is added to w's momentum on stream `here`."""
        self.here = here
        self.waits.clear()
        opt.accumulate_grad(w)
        return list(self.waits)


def test_sums_on_several_streams_follow_each_other(monkeypatch):
    w, v = (torch.randn(4, 5, requires_grad=True) for _ in range(2))
    opt, s = d3.Dion3([w, v]), Streams(monkeypatch)
    assert s.sums(opt, w, "a") == []                  # (its zeros were made there)
    assert s.sums(opt, w, "b") == [("b", "a")]        # behind the first sum and the zeros
    assert s.sums(opt, w, "b") == []
    assert s.sums(opt, v, "c") == []                  # another buffer
    assert s.sums(opt, w, "c") == [("c", "b")]
    assert opt._streams == {"c"}
    s.here = "d"
    s.waits.clear()
    opt.momentum(w)                                   # a reader
    assert s.waits == [("d", "c")]
    assert s.sums(opt, w, "a") == [("a", "d")]


def test_captured_sums_follow_captured_ones_only(monkeypatch):
    w = torch.randn(4, 5, requires_grad=True)
    opt, s = d3.Dion3([w]), Streams(monkeypatch)
    s.sums(opt, w, "a")
    s.captured = {"c", "d"}
    assert s.sums(opt, w, "c") == []                  # cannot wait for work outside
    assert s.sums(opt, w, "d") == [("d", "c")]
    s.captured = set()
    assert s.sums(opt, w, "b") == [("b", "a")]        # nor is the capture work to wait for
    s.captured = {"e"}
    assert s.sums(opt, w, "e") == []                  # another capture


def test_captures_name_no_parameters(monkeypatch):
    """Capturing a backward pass adds nothing yet, so the next step has nothing to step."""
    w = torch.randn(4, 5, requires_grad=True)
    opt, s = d3.Dion3([w]), Streams(monkeypatch)
    opt.momentum(w)
    s.captured = {"c"}
    s.sums(opt, w, "c")
    assert not opt._accumulated and not opt._streams
    s.captured = set()
    s.sums(opt, w, "a")                               # before a replay
    assert w in opt._accumulated and opt._streams == {"a"}


def test_refused_product_names_no_parameter(monkeypatch):
    """A weight gradient that raises (no memory, a stride past the limit) has
    added nothing, so a step that follows all the same leaves w alone."""
    x, w, _, dy, opt, y = setting()

    def refuse(dz, x, out=None, accumulate=False):
        raise d3.Dion3Error(-3, "dion3_linear_grad_weight")

    with monkeypatch.context() as mp:
        mp.setattr(layer, "linear_grad_weight", refuse)
        with pytest.raises(d3.Dion3Error):
            y.backward(dy, retain_graph=True)
    assert untouched(opt, w)
    y.backward(dy)
    assert w in opt._accumulated


def test_loaded_state_holds_no_pending_gradient(monkeypatch):
    x, w, _, dy, opt, y = setting()
    opt.momentum(w).fill_(3)
    saved = copy.deepcopy(opt.state_dict())           # as read from a file
    y.backward(dy)
    assert w in opt._accumulated
    s = Streams(monkeypatch)
    s.here = "b"
    opt.load_state_dict(saved)
    assert not opt._accumulated and (opt.momentum(w) == 3).all()
    assert s.sums(opt, w, "c") == [("c", "b")]        # behind the load


def test_gradients_of_any_layout():
    """What the library cannot read in place is copied: no rows, or rows past its stride limit."""
    t = torch.randn(3, 8)
    assert layer._as_rows(t) is t
    wide = torch.empty(2, (1 << 21) + 8, dtype=torch.bfloat16)
    for v in (wide[:, :8], t.t(), t[:1].expand(4, 8), torch.ones(()).expand(3, 8)):
        c = layer._as_rows(v)
        assert c.is_contiguous() and c.data_ptr() != v.data_ptr() and c.shape == v.shape
    v = wide[:, 8:].as_strided((2, 8), (1 << 21, 1))
    assert layer._as_rows(v) is v


def test_step_follows_every_momentum_it_takes(monkeypatch):
    """One wait a stream; each buffer last used elsewhere is held for the step's stream."""
    ws = [torch.randn(4, 5, requires_grad=True) for _ in range(4)]
    opt, s = d3.Dion3(ws), Streams(monkeypatch)
    monkeypatch.setattr(optim._lib, "Group", lambda *a, **k: None)
    monkeypatch.setattr(optim._lib, "step_groups", lambda *a, **k: None)
    s.sums(opt, ws[0], "b")
    s.sums(opt, ws[1], "b")
    s.sums(opt, ws[2], "c")
    ws[3].grad = torch.ones_like(ws[3])
    s.here = "a"
    s.waits.clear()
    s.held.clear()
    opt.step()
    assert s.waits == [("a", "b"), ("a", "c")]
    assert [(t is opt.state[w]["momentum"], at) for (t, at), w in zip(s.held, ws)] == [(True, "a")] * 3
    assert not opt._accumulated and not opt._streams
    assert s.sums(opt, ws[0], "b") == [("b", "a")]    # behind the step
    assert s.sums(opt, ws[3], "b") == [("b", "a")]


def test_hooks_see_no_gradient():
    """A summed gradient passes by w's hooks, which run with None and without a .grad."""
    x, w, _, dy, opt, y = setting()
    seen = []
    w.register_hook(lambda g: seen.append(("hook", g)))
    w.register_post_accumulate_grad_hook(lambda p: seen.append(("post", p.grad)))
    y.backward(dy)
    assert seen == [("hook", None), ("post", None)]
    assert torch.equal(opt.momentum(w), dy.t() @ x.detach())
