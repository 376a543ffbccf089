"""The differentiable layer operators as a model uses them, and the optimizer
that takes weight gradients straight into its momentum."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import U, d

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def rnd(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def params(seed, hidden=264, mlp=520):
    g = torch.Generator().manual_seed(seed)
    p = {"n1": 1 + rnd(g, hidden, std=0.1), "w1": rnd(g, mlp, hidden, std=0.06),
         "b1": rnd(g, mlp, std=0.1), "w2": rnd(g, hidden, mlp, std=0.04),
         "b2": rnd(g, hidden, std=0.1)}
    return {k: v.requires_grad_(True) for k, v in p.items()}


def block(p, x, r, checkpoint="f8", into=None):
    """norm -> linear, activation -> linear onto the residual stream."""
    y, h, packed = d3.rms_norm_residual(x, p["n1"], residual=r, pack=checkpoint == "f8")
    a = d3.linear_layer(y, p["w1"], p["b1"], act="gelu_tanh", into=into,
                        checkpoint=packed if checkpoint == "f8" else "full")
    return d3.linear_layer(a, p["w2"], p["b2"], residual=h, checkpoint=checkpoint, into=into)


def data(seed, *lead, hidden=264, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return [rnd(g, *lead, hidden, dtype=dtype) for _ in range(3)]


def plain(p, x, r, dout, dtype):
    """The block's gradients by the formulas in 64 bits (no rounding inside)."""
    q = {k: d(v).requires_grad_(True) for k, v in p.items()}
    xd, rd = d(x).requires_grad_(True), d(r).requires_grad_(True)
    h = xd + rd
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * q["n1"]
    a = torch.nn.functional.gelu(y @ q["w1"].T + q["b1"], approximate="tanh")
    out = a @ q["w2"].T + q["b2"] + h
    out.backward(d(dout))
    return out.detach(), {**{k: v.grad for k, v in q.items()}, "x": xd.grad, "r": rd.grad}


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("checkpoint", ["full", "f8"])
@pytest.mark.parametrize("lead", [(1,), (37,), (4, 75)])
def test_block_gradients(lead, checkpoint, dtype):
    """Against the formulas: each tensor that passes between operators is
    rounded once to the 16-bit type (fewer than 8 roundings on any path, each
    at most U relative), and with 8-bit checkpoints the inputs of the weight
    gradients and of the activation's slope are off by at most 2^-4 of
    themselves; both in the norm, where independent roundings only shrink."""
    p = params(1)
    x, r, dout = data(2, *lead, dtype=dtype)
    x.requires_grad_(True)
    r.requires_grad_(True)
    out = block(p, x, r, checkpoint)
    out.backward(dout)
    want, grads = plain(p, x, r, dout, dtype)
    rel = float((d(out) - want).norm() / want.norm())
    assert rel <= 8 * U[dtype], rel
    for k, t in {**p, "x": x, "r": r}.items():
        assert t.grad.dtype == t.dtype
        e = float((d(t.grad) - grads[k]).norm() / grads[k].norm())
        assert e <= 8 * U[dtype] + (2 ** -4 if checkpoint == "f8" else 0), (k, e)


def test_block_is_its_operators():
    """Autograd adds nothing of its own: the same bits as the operators called by hand."""
    p = params(3)
    x, r, dout = data(4, 90)
    x.requires_grad_(True)
    r.requires_grad_(True)
    block(p, x, r).backward(dout)
    with torch.no_grad():
        w1, w2 = p["w1"].to(BF), p["w2"].to(BF)
        y, h, rstd, py = d3.add_rms_norm(x, p["n1"], residual=r, pack=True)
        a, z = d3.linear(y, w1, p["b1"], act="gelu_tanh", return_preact=True)
        pz, pa = d3.pack_f8(z), d3.pack_f8(a)
        dw2, db2 = d3.linear_grad_weight(dout, pa), d3.act_grad(dout, None, "none", bias=True)[1]
        da = d3.linear_grad_input(dout, w2)
        dz, db1 = d3.act_grad(da, pz, "gelu_tanh", bias=True)
        dw1 = d3.linear_grad_weight(dz, py)
        dx, dn = d3.add_rms_norm_grad(d3.linear_grad_input(dz, w1), h, rstd, p["n1"], dh=dout)
    for got, want in ((p["w2"].grad, dw2), (p["b2"].grad, db2), (p["w1"].grad, dw1),
                      (p["b1"].grad, db1), (p["n1"].grad, dn), (x.grad, dx), (r.grad, dx)):
        assert torch.equal(got, want)


def test_partial_gradients():
    """Only what asks for a gradient gets one; unused outputs cost none."""
    p = params(5)
    x, r, dout = data(6, 33)
    for name in ("w1", "b2", "n1"):
        q = {k: v.detach().requires_grad_(k == name) for k, v in p.items()}
        block(q, x, r).backward(dout)
        full = {k: v.detach().requires_grad_(True) for k, v in p.items()}
        block(full, x, r).backward(dout)
        for k in q:
            assert (q[k].grad is not None) == (k == name)
        assert torch.equal(q[name].grad, full[name].grad)
    x.requires_grad_(True)
    y, h, _ = d3.rms_norm_residual(x, p["n1"], residual=r)
    h.backward(dout)                          # past the norm only
    assert torch.equal(x.grad, dout) and p["n1"].grad is None
    x.grad = None
    y, h, _ = d3.rms_norm_residual(x, p["n1"].detach())
    y.backward(dout)                          # no residual
    want = d3.add_rms_norm_grad(dout, x.detach(), d3.add_rms_norm(x.detach(), p["n1"].detach())[2],
                                p["n1"].detach())[0]
    assert torch.equal(x.grad, want)
    x.grad = None
    y, h, _ = d3.rms_norm_residual(x, p["n1"].detach())
    torch.autograd.backward([y, h], [dout, dout])          # x itself is the stream that goes on
    want = d3.add_rms_norm_grad(dout, x.detach(), d3.add_rms_norm(x.detach(), p["n1"].detach())[2],
                                p["n1"].detach(), dh=dout)[0]
    assert torch.equal(x.grad, want)
    with torch.no_grad():
        assert not block(p, x, r).requires_grad


def test_broadcast_and_transposed_gradients():
    """An expanded gradient (of a sum), a transposed one, and one of a shared weight."""
    p = params(7)
    x, r, _ = data(8, 3, 20)
    x.requires_grad_(True)
    out = block(p, x, r)
    out.float().sum().backward()
    a = {k: v.grad.clone() for k, v in p.items()}
    gx = x.grad.clone()
    for v in (*p.values(), x):
        v.grad = None
    block(p, x, r).backward(torch.ones_like(out))
    for k, v in p.items():
        assert torch.equal(a[k], v.grad)
    assert torch.equal(gx, x.grad)
    # through a transpose
    for v in (*p.values(), x):
        v.grad = None
    t = torch.randn(3, 264, 20, device="cuda").to(BF)
    block(p, x, r).transpose(1, 2).backward(t)
    b = p["w2"].grad.clone()
    p["w2"].grad = None
    block(p, x, r).backward(t.transpose(1, 2).contiguous())
    assert torch.equal(b, p["w2"].grad)
    # one weight used twice: the gradients add up
    w = torch.randn(264, 264, device="cuda").mul_(0.05).requires_grad_(True)
    dy = torch.randn(3, 20, 264, device="cuda").to(BF)
    y1 = d3.linear_layer(x.detach(), w)
    d3.linear_layer(y1, w).backward(dy)
    g2 = d3.linear_grad_weight(dy, d3.pack_f8(y1.detach()))
    g1 = d3.linear_grad_weight(d3.linear_grad_input(dy, w.detach().to(BF)), d3.pack_f8(x.detach()))
    assert torch.allclose(w.grad, g1 + g2, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("normalize", [False, True])
def test_optimizer_takes_gradients_into_its_momentum(normalize):
    """Steps with gradients summed into the momentum equal steps on .grad: the
    first bit for bit (0 + dW), the later ones too, since each adds one fp32
    gradient to M once."""
    runs = []
    for direct in (False, True):
        p = params(9)
        opt = d3.Dion3([p["w1"], p["w2"]], lr=0.02, fraction=0.25, normalize=normalize)
        for k in range(3):
            x, r, dout = data(20 + k, 150)
            block(p, x, r, into=opt if direct else None).backward(dout)
            assert (p["w1"].grad is None) == direct
            opt.step()
            for v in p.values():
                v.grad = None
        runs.append([p["w1"].detach(), p["w2"].detach(), opt.momentum(p["w1"]),
                     opt.momentum(p["w2"])])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_momentum_accumulates_over_backward_passes():
    """Two backward passes before a step; a .grad beside the summed gradient;
    nothing new: no step."""
    p = params(10)
    opt = d3.Dion3([p["w1"], p["w2"]], lr=0.02, fraction=0.25)
    x, r, dout = data(11, 64)
    for _ in range(2):
        block(p, x, r, into=opt).backward(dout)
    m2 = opt.momentum(p["w1"]).clone()
    q = params(10)
    block(q, x, r).backward(dout)
    assert torch.equal(m2, q["w1"].grad + q["w1"].grad)
    p["w1"].grad = q["w1"].grad.clone()
    w0, v0 = p["w1"].detach().clone(), p["w2"].detach().clone()
    ref_w, ref_m = w0.clone(), m2.clone()
    d3.step(ref_w, ref_m, d3.k_from_fraction(0.25, 520), 0.02 / 0.5, 0.95, G=p["w1"].grad)
    opt.step()
    assert torch.equal(p["w1"].detach(), ref_w) and torch.equal(opt.momentum(p["w1"]), ref_m)
    assert not torch.equal(p["w2"].detach(), v0)
    p["w1"].grad = None
    w1, m1 = p["w1"].detach().clone(), opt.momentum(p["w1"]).clone()
    opt.step()                                  # nothing accumulated since
    assert torch.equal(p["w1"].detach(), w1) and torch.equal(opt.momentum(p["w1"]), m1)


def test_step_waits_for_the_stream_of_the_backward_pass():
    """Forward on a side stream, backward and step from the default one: the
    weight gradients, which autograd never sees, are summed before the step
    reads them."""
    def fresh():
        p = params(15, 1024, 4096)
        return p, d3.Dion3([p["w1"], p["w2"]], lr=0.02, fraction=0.25)

    x, r, dout = data(16, 8192, hidden=1024)
    p, opt = fresh()
    block(p, x, r, into=opt).backward(dout)
    opt.step()
    want = [p["w1"].detach().clone(), opt.momentum(p["w1"]).clone()]
    p, opt = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = d3.linear_layer(x, p["w1"], into=opt)      # (allocations and first launches)
        out = block(p, x, r, into=opt)
    torch.cuda.current_stream().wait_stream(side)
    out.backward(dout)
    assert side in opt._streams
    opt.step()
    assert not opt._streams and not opt._accumulated
    assert torch.equal(p["w1"].detach(), want[0]) and torch.equal(opt.momentum(p["w1"]), want[1])


def test_training_step_in_a_graph():
    """Forward, backward into the momentum and the optimizer's step as one
    captured graph: every replay equals the eager step."""
    def one(p, opt, x, r, dout):
        block(p, x, r, into=opt).backward(dout)
        for v in p.values():
            v.grad = None
        opt.step()

    def fresh():
        p = params(12)
        return p, d3.Dion3([p["w1"], p["w2"]], lr=0.02, fraction=0.25)

    batches = [data(30 + k, 96) for k in range(4)]
    p, opt = fresh()
    want = []
    for b in batches:
        one(p, opt, *b)
        want.append([p["w1"].detach().clone(), p["w2"].detach().clone(),
                     opt.momentum(p["w1"]).clone()])
    p, opt = fresh()
    w0 = [p["w1"].detach().clone(), p["w2"].detach().clone()]
    x, r, dout = (t.clone() for t in batches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):               # allocations and first launches
        one(p, opt, x, r, dout)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(p, x, r, into=opt).backward(dout)
    step = [d3.Group([p[k].detach()], [opt.momentum(p[k])], d3.k_from_fraction(0.25, p[k].shape[0]),
                     0.02 / 0.5) for k in ("w1", "w2")]
    with torch.no_grad():
        p["w1"].copy_(w0[0])
        p["w2"].copy_(w0[1])
        opt.momentum(p["w1"]).zero_()
        opt.momentum(p["w2"]).zero_()
    for b, w in zip(batches, want):
        for dst, src in zip((x, r, dout), b):
            dst.copy_(src)
        graph.replay()
        d3.step_groups(step, 0.95)              # eager work between the replays
        torch.cuda.synchronize()
        got = [p["w1"].detach(), p["w2"].detach(), opt.momentum(p["w1"])]
        for u, v in zip(got, w):
            assert torch.equal(u, v)


def test_momentum_is_not_made_in_a_capture(monkeypatch):
    """The momentum's zeros would be part of the graph, and every replay would
    start from them.  (Only the answer to whether a capture runs is forced.)"""
    p = params(17)
    x, _, _ = data(18, 8)
    opt = d3.Dion3([p["w1"], p["w2"]])
    opt.momentum(p["w2"])
    with monkeypatch.context() as mp:
        mp.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError):
            d3.linear_layer(x, p["w1"], into=opt)
        with pytest.raises(RuntimeError):
            opt.accumulate_grad(p["w1"])
        assert not opt.state[p["w1"]] and not opt._accumulated and not opt._streams
        assert opt.accumulate_grad(p["w2"]) is opt.momentum(p["w2"])
    with pytest.raises(ValueError):
        opt.accumulate_grad(x)
    d3.linear_layer(x, p["w1"], into=opt)


def test_refusals():
    p = params(13)
    x, r, _ = data(14, 8)
    opt = d3.Dion3([p["w1"]])
    with pytest.raises(ValueError):
        d3.linear_layer(x, p["w2"], into=opt)                        # not its parameter
    with pytest.raises(ValueError):
        d3.linear_layer(x, p["w1"], checkpoint="f16")
    with pytest.raises(ValueError):
        d3.linear_layer(x, p["w1"], checkpoint=d3.pack_f8(x[:4]))
    with pytest.raises(TypeError):
        d3.linear_layer(x, p["w1"].detach().half())
    with pytest.raises(TypeError):
        d3.linear(x, p["w1"].detach())                               # fp32 weights
    with pytest.raises(ValueError):
        d3.linear(x, p["w2"].detach().to(BF))                        # wrong width
    with pytest.raises(ValueError):
        d3.linear(x, p["w1"].detach().to(BF), act="tanh")
    with pytest.raises(ValueError):
        d3.linear(x.t(), p["w1"].detach().to(BF))                    # strided features
    with pytest.raises(ValueError):
        d3.linear(x[:1].expand(8, -1), p["w1"].detach().to(BF))      # overlapping rows
    with pytest.raises(ValueError):
        d3.linear_grad_weight(x, x, accumulate=True)
    with pytest.raises(ValueError):
        d3.linear_grad_weight(x, x[:4])
    with pytest.raises(ValueError):
        d3.linear_grad_weight(x, x, out=torch.zeros(3, 3, device="cuda"))
    with pytest.raises(TypeError):
        d3.linear_grad_weight(x, x, out=torch.zeros(264, 264, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        d3.add_rms_norm(x, p["n1"].detach(), residual=r[:4])
    with pytest.raises(ValueError):
        d3.add_rms_norm(x, p["n1"].detach(), return_y=False)
    with pytest.raises(TypeError):
        d3.add_rms_norm(x, p["n1"].detach().half())
    with pytest.raises(TypeError):
        d3.add_rms_norm(x.float(), p["n1"].detach())
    with pytest.raises(d3.Dion3Error):
        d3.add_rms_norm(x, p["n1"].detach(), eps=-1.0)
    with pytest.raises(TypeError):
        d3.act_grad(x, x.half(), "silu")
    with pytest.raises(ValueError):
        d3.act_grad(x, d3.pack_f8(x[:4]), "silu")
    with pytest.raises(ValueError):
        d3.PackedF8(d3.pack_f8(x).q, d3.pack_f8(x).scale, 300)
