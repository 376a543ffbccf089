"""A whole training step made of the package's operators: tokens, embedding,
norm, projections, heads' norm and rotation, attention (plain, in fp32), mlp,
head, log probabilities, backward, clipping, the optimizer's step."""
import functools
import math

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, U, d

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
V, C, H, HK, D, MLP = 203, 96, 4, 2, 24, 200
FREQS = 10000.0 ** (-torch.arange(0, 16, 2, dtype=torch.float64) / 16)


@functools.lru_cache
def device_freqs():
    return FREQS.cuda()


def params(seed):
    g = torch.Generator().manual_seed(seed)

    def w(*shape, std=0.08):
        return torch.randn(shape, generator=g) * std

    p = {"emb": w(V, C, std=0.3), "n1": 1 + w(C), "wqkv": w((H + 2 * HK) * D, C), "nq": 1 + w(D),
         "nk": 1 + w(D), "wo": w(C, H * D), "n2": 1 + w(C), "w1": w(MLP, C), "w2": w(C, MLP),
         "nf": 1 + w(C), "head": w(V, C)}
    return {k: v.cuda().requires_grad_(True) for k, v in p.items()}


MATRICES = ("wqkv", "wo", "w1", "w2")


def attend(q, k, v):
    """Causal attention [B, S, heads, D] in q's precision, keys shared by groups of heads."""
    k, v = (t.repeat_interleave(q.shape[2] // k.shape[2], 2) for t in (k, v))
    q, k, v = (t.transpose(1, 2).contiguous() for t in (q, k, v))
    s = (q.unsqueeze(3) * k.unsqueeze(2)).sum(-1) / math.sqrt(q.shape[-1])
    S = q.shape[2]
    s = s.masked_fill(torch.ones(S, S, device=q.device).triu(1).bool(), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return (p.unsqueeze(-1) * v.unsqueeze(2)).sum(3).transpose(1, 2)


def model(p, tokens, into=None):
    """Logits [B, S, V]."""
    B, S = tokens.shape
    pos, freqs = torch.arange(S, device="cuda"), device_freqs()
    x = d3.embedding_layer(tokens, p["emb"], scale=math.sqrt(C) / 4, dtype=BF)
    y, h, _ = d3.rms_norm_residual(x, p["n1"])
    qkv = d3.linear_layer(y, p["wqkv"], checkpoint="full", into=into)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split((H * D, HK * D, HK * D), -1))
    q, k = d3.qk_norm_rope_layer(q, k, p["nq"], p["nk"], pos, freqs)
    a = attend(q.float(), k.float(), v.float()).to(BF).reshape(B, S, H * D)
    o = d3.linear_layer(a, p["wo"], checkpoint="full", into=into)
    y, h, _ = d3.rms_norm_residual(o, p["n2"], residual=h)
    z = d3.linear_layer(y, p["w1"], act="silu", checkpoint="full", into=into)
    h = d3.linear_layer(z, p["w2"], residual=h, checkpoint="full", into=into)
    y, _, _ = d3.rms_norm_residual(h, p["nf"])
    return d3.linear_layer(y, p["head"], checkpoint="full")


def loss_of(logits, targets, bonus=0.01):
    logp, entropy = d3.token_log_probs(logits, targets, scale=0.9, entropy=True)
    return -(logp.sum() + bonus * entropy.sum()) / targets.numel()


def plain(p, tokens, targets, bonus=0.01):
    """(loss, gradients) by the formulas in 64 bits."""
    q = {k: d(v).requires_grad_(True) for k, v in p.items()}

    def norm(t, w):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w

    def turn(t):
        ang = (torch.arange(t.shape[1]).double()[:, None] * FREQS)[:, None]
        c, s = torch.cos(ang), torch.sin(ang)
        a, b, rest = t[..., :8], t[..., 8:16], t[..., 16:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)

    B, S = tokens.shape
    h = q["emb"][tokens.cpu()] * (math.sqrt(C) / 4)
    qkv = norm(h, q["n1"]) @ q["wqkv"].T
    a, b, v = (t.unflatten(-1, (-1, D)) for t in qkv.split((H * D, HK * D, HK * D), -1))
    o = attend(turn(norm(a, q["nq"])), turn(norm(b, q["nk"])), v).reshape(B, S, H * D)
    h = h + o @ q["wo"].T
    h = h + torch.nn.functional.silu(norm(h, q["n2"]) @ q["w1"].T) @ q["w2"].T
    lp = torch.log_softmax(0.9 * (norm(h, q["nf"]) @ q["head"].T), -1)
    t = targets.cpu()
    got = torch.where(t >= 0, lp.gather(-1, t.clamp_min(0)[..., None])[..., 0], 0.0)
    loss = -(got.sum() - bonus * (lp.exp() * lp).sum()) / t.numel()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in q.items()}


def batch(seed, B=3, S=21):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (B, S + 1), generator=g)
    t[0, :4] = 7                                              # a frequent token
    tokens, targets = t[:, :-1].contiguous(), t[:, 1:].contiguous()
    targets[1, -5:] = -100                                    # padding
    return tokens.cuda(), targets.cuda()


def test_loss_and_gradients():
    """Against the formulas: what passes between operators is rounded to bf16
    (about 20 roundings on the longest path, each at most U of its tensor, and
    norms of independent roundings only shrink)."""
    p = params(1)
    tokens, targets = batch(2)
    loss = loss_of(model(p, tokens), targets)
    loss.backward()
    want, grads = plain(p, tokens, targets)
    assert abs(float(loss.detach()) - float(want)) <= 20 * U[BF] * abs(float(want))
    for k, v in p.items():
        assert v.grad.dtype == v.dtype and v.grad.shape == v.shape
        e = float((d(v.grad) - grads[k]).norm() / grads[k].norm())
        assert e <= 20 * U[BF], (k, e)


def test_clipped_steps():
    """Gradients of all parameters clipped by one norm, then the optimizer's
    step for the matrices: the same as scaling by hand; and three steps run."""
    p = params(3)
    opt = d3.Dion3([p[k] for k in MATRICES], lr=0.01)
    rest = [v for k, v in p.items() if k not in MATRICES]
    for step in range(3):
        tokens, targets = batch(10 + step)
        for v in p.values():
            v.grad = None
        loss = loss_of(model(p, tokens), targets)
        loss.backward()
        raw = {k: d(v.grad) for k, v in p.items()}
        before = {k: d(opt.momentum(p[k])) for k in MATRICES}
        total = math.sqrt(sum(float((g * g).sum()) for g in raw.values()))
        most = float(torch.tensor(total / 3))
        norm = d3.clip_grad_norm([v.grad for v in p.values()], most)
        assert abs(float(norm) - total) <= total * EPS32 * 1.001
        for k, v in p.items():
            w = raw[k] * most / total
            assert (d(v.grad) - w).abs().max() <= w.abs().max() * EPS32 * 1.001
        clipped = {k: d(p[k].grad) for k in MATRICES}
        opt.step()
        for k in MATRICES:                                    # M + clipped, the selected rows decayed
            m, s = d(opt.momentum(p[k])), before[k] + clipped[k]
            assert (torch.minimum((m - s).abs(), (m - 0.95 * s).abs()) <= 4 * EPS32 * s.abs() + 1e-12).all()
        with torch.no_grad():
            for v in rest:
                v -= 0.1 * v.grad
        assert math.isfinite(float(loss.detach()))


def test_16_bit_gradients_clipped_into_the_momenta():
    """A copy of the weights in bf16 carries the gradients; they are clipped and
    summed into the momenta of the fp32 weights."""
    p = params(4)
    opt = d3.Dion3([p[k] for k in MATRICES])
    low = {k: (v.detach().to(BF).requires_grad_(True) if k in MATRICES else v) for k, v in p.items()}
    tokens, targets = batch(5)
    loss_of(model(low, tokens), targets).backward()
    grads = [low[k].grad for k in MATRICES]
    assert all(t.dtype == BF for t in grads)
    norm = d3.grad_norm(grads)
    d3.clip_grad_norm(grads, float(norm) / 2, into=[opt.accumulate_grad(p[k]) for k in MATRICES])
    for k, t in zip(MATRICES, grads):
        w = d(t) * (float(norm) / 2 / float(d3.grad_norm(grads)))
        assert ((d(opt.momentum(p[k])) - w).abs() <= w.abs() * 3 * EPS32).all()
    before = {k: p[k].detach().clone() for k in MATRICES}
    opt.step()
    assert all(not torch.equal(before[k], p[k]) and torch.isfinite(p[k]).all() for k in MATRICES)


def test_captured_step():
    """Forward, backward and clipping in one graph: every replay equals the eager pass."""
    p = params(6)
    tokens, targets = batch(7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def run(q):
        for v in q.values():
            v.grad = None
        loss = loss_of(model(q, tokens), targets)
        loss.backward()
        norm = d3.clip_grad_norm([v.grad for v in q.values()], 0.5)
        return loss.detach(), norm

    with torch.cuda.stream(s):
        for _ in range(2):
            run(p)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        loss, norm = run(p)
    static = {k: v.grad for k, v in p.items()}
    for k in range(3):
        a, b = batch(20 + k)
        tokens.copy_(a)
        targets.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        q = {n: v.detach().clone().requires_grad_(True) for n, v in p.items()}
        el, en = run(q)
        # (the attention and the loss are torch's; the norm is over the package's gradients)
        assert abs(float(loss) - float(el)) <= 1e-6 * abs(float(el))
        assert abs(float(norm) - float(en)) <= 1e-5 * float(en)
        for n in q:
            e = float((d(static[n]) - d(q[n].grad)).norm() / d(q[n].grad).norm())
            assert e <= 1e-5, (n, e)
