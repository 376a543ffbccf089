"""Random sizes, strides, alignments, types and masks of the embedding, the
heads' norm and rotation, the log probabilities and the clipping against the
64-bit formulas, with NaN around the operands and workspaces that are exactly
as long as asked for, hold other numbers before and guard bytes behind."""
import math
import random

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests import test_gpu_clip as clip
from tests import test_gpu_embedding as emb
from tests import test_gpu_heads as heads
from tests import test_gpu_log_probs as logp
from tests.layer_ref import EPS32, TINY, U, close, rounded
from tests.test_gpu_layer_fuzz import place, size

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
SEEDS = range(24)


class Exact:
    """A workspace of exactly the bytes asked for."""

    def __init__(self):
        self.bufs = []

    def get(self, nbytes, device):
        buf = torch.randint(0, 256, (nbytes + 1280,), dtype=torch.uint8, device=device)
        off = (-buf.data_ptr()) % 256
        buf[off + nbytes:] = 0xA5
        self.bufs.append((buf, off + nbytes))
        return buf.data_ptr() + off, nbytes

    def check(self, what):
        for buf, end in self.bufs:
            assert (buf[end:] == 0xA5).all(), what


def near(r, v):
    """v, or a size next to it."""
    return max(1, v + r.choice([-1, 0, 0, 1]))


@pytest.mark.parametrize("seed", SEEDS)
def test_random_embeddings(seed):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    for _ in range(3):
        T = r.choice([size(r, 3000), near(r, 64), near(r, 8192), size(r, 40000)])
        m = r.choice([size(r, 3000), near(r, 512), near(r, 4)])
        m = min(m, max(1, 3000000 // T))
        n = min(size(r, 60000), max(1, 3000000 // m))
        kind, t = r.choice(emb.KINDS), r.choice([BF, FP, F32])
        what = (seed, T, n, m, kind, t)
        tokens, dy = emb.text(g, T, n, kind), emb.rnd(g, T, m, dtype=t)
        tokens = tokens if r.random() < 0.5 else tokens.int()
        ok = (tokens >= 0) & (tokens < n)
        dy[~ok] = r.choice([0.0, math.nan])                  # a padded place's is not read into a sum
        want, off = emb.grad(tokens, dy, n, 1.0)
        ws = Exact()
        out = place(r, torch.zeros(n, m, device="cuda"))
        buf = out._base if out._base is not None else out
        keep = buf.clone()
        d3.embedding_grad(tokens.cuda(), place(r, dy.cuda()), n, out=out, ws=ws)
        close(out, want, off, what)
        have = torch.zeros(n, dtype=torch.bool)
        have[tokens[ok].long()] = True
        out.copy_(torch.where(have[:, None], 1.0, math.nan))
        d3.embedding_grad(tokens.cuda(), place(r, dy.cuda()), n, out=out, accumulate=True, ws=ws)
        lim = off + (want + 1).abs() * EPS32
        close(out[have.cuda()], want[have] + 1, lim[have], what)
        assert torch.isnan(out.cpu()[~have]).all(), what
        ws.check(what)
        out.copy_(keep.as_strided(out.shape, out.stride(), out.storage_offset()))
        assert torch.equal(buf.view(torch.int32), keep.view(torch.int32)), what    # nothing around it
        w = emb.rnd(g, n, m, dtype=t)
        y = d3.embedding(tokens.cuda(), place(r, w.cuda()))
        assert torch.equal(y.cpu(), torch.where(ok[:, None], w[tokens.clamp(0, n - 1).long()], 0)), what


def laid(r, t):
    """t [T, heads, D] with NaN around it: contiguous, rows apart, heads first,
    at any element."""
    T, h, D = t.shape
    off, gap = r.choice([0, 0, 1, 8]), r.choice([0, 0, 1, 8, 13])
    how = r.choice(["tokens", "heads"])
    hs = D + gap if how == "tokens" else (D + gap) * T + gap
    ld = h * hs + gap if how == "tokens" else D + gap
    buf = torch.full((h * hs + T * ld + off + 64,), math.nan, dtype=t.dtype, device="cuda")
    v = buf.as_strided((T, h, D), (ld, hs, 1), off)
    v.copy_(t)
    return v


@pytest.mark.parametrize("seed", SEEDS)
def test_random_heads(seed):
    r, g = random.Random(100 + seed), torch.Generator().manual_seed(seed)
    for _ in range(3):
        D = r.choice([16 * r.randint(1, 20), r.randint(1, 300), 128])
        rot = r.choice([D // 2 * 2, 2 * r.randint(0, D // 2), min(D, 16 * r.randint(0, 4)) // 2 * 2])
        T = r.choice([size(r, 600), size(r, 40)])
        hq, hk = r.randint(1, 40), r.choice([1, 2, 8, r.randint(1, 20)])
        if T * hq * D > 400000:
            T = max(1, 400000 // (hq * D))
        t, il, eps = r.choice([BF, FP]), r.random() < 0.5, r.choice([1e-6, 1e-5])
        what = (seed, T, hq, hk, D, rot, t, il)
        wtype = r.choice([t, F32])
        q, k, wq, wk, fr = heads.inputs(g, T, hq, hk, D, rot, t, wtype)
        pos = torch.randint(-50, 100000, (T,), generator=g)
        pos = pos if r.random() < 0.5 else pos.int()
        dyq, dyk = heads.rnd(g, T, hq, D, dtype=t), heads.rnd(g, T, hk, D, dtype=t)
        args = (laid(r, q), laid(r, k), wq.cuda(), wk.cuda(), pos.cuda(), fr.cuda())
        yq, yk = d3.qk_norm_rope(*args, eps=eps, interleaved=il)
        ws = Exact()
        dq, dk, dwq, dwk = d3.qk_norm_rope_grad(laid(r, dyq), laid(r, dyk), *args, eps=eps, interleaved=il,
                                                ws=ws)
        ws.check(what)
        for x, w, y, dy, dx, dw in ((q, wq, yq, dyq, dq, dwq), (k, wk, yk, dyk, dk, dwk)):
            want, big = heads.formula(x, w, pos, fr, il, eps)
            close(y, want, rounded(want, t, big * (heads.CHAIN / 2 + heads.TURN + 4) * EPS32), what)
            wx, lim, ww, wl = heads.grad_formula(dy, x, w, pos, fr, il, eps)
            close(dx, wx, rounded(wx, t, lim * (2 * heads.CHAIN + heads.TURN + 8) * EPS32), what)
            n = x.shape[0] * x.shape[1]
            close(dw, ww, wl * (n + heads.CHAIN + heads.TURN) * EPS32 + 1e-30, what)


@pytest.mark.parametrize("seed", SEEDS)
def test_random_log_probs(seed):
    r, g = random.Random(200 + seed), torch.Generator().manual_seed(seed)
    for _ in range(3):
        n = r.choice([size(r, 3000), size(r, 300000), near(r, 8192), near(r, 131072)])
        T = min(size(r, 300), max(1, 500000 // n))
        t, scale = r.choice(logp.DTYPES), r.choice([1.0, 0.5, 1.25])
        what = (seed, T, n, t, scale)
        x = logp.logits(g, T, n, t, r.choice([0.5, 3.0, 20.0]))
        if r.random() < 0.4:                                  # masked, one logit a row stays
            at = torch.randint(0, n, (T, 1), generator=g)
            stay = x.gather(1, at)
            x[torch.rand(T, n, generator=g) < r.choice([0.3, 0.999])] = -math.inf
            x.scatter_(1, at, stay)
        targets = torch.randint(-1, n + 1, (T,), generator=g)
        top = r.choice([0, 1, min(n, r.randint(1, 64)), min(n, 64)])
        w = logp.Want(x, targets, scale)
        ws, X = Exact(), place(r, x.cuda())
        lp, stats, H, tl, ti = d3.log_probs(X, targets.cuda(), scale=scale, entropy=True, top=top, ws=ws)
        ws.check(what)
        masked = torch.isinf(w.logp)
        assert (lp.cpu()[masked] == -math.inf).all(), what
        close(lp[~masked.cuda()], w.logp[~masked], w.logp_off[~masked], what)
        close(H, w.H, w.H_off, what)
        if top:
            at = logp.best(x, top)
            assert torch.equal(ti.cpu(), at), what
            want = w.q.gather(1, at)
            got, off = tl.cpu().double(), w.l_off[:, None] + (w.dz.gather(1, at).abs() + want.abs()) * EPS32
            low = torch.isinf(want)
            assert (got[low] == -math.inf).all(), what
            assert ((got - want).abs()[~low] <= off[~low]).all(), what
        gl, gh = torch.randn(T, generator=g), torch.randn(T, generator=g) if r.random() < 0.5 else None
        dx = d3.log_probs_grad(gl.cuda(), X, targets.cuda(), stats, scale=scale, entropy=H,
                               dentropy=None if gh is None else gh.cuda())
        want, off = w.grad(gl, gh, scale)
        # a probability below 2^-126 may count as none: what its factor, g + gH
        # (|ln p| + H) times the scale, makes of 2^-126
        lnp = w.q.abs().clamp_max(110)                        # (below e^-110 the value itself is less)
        lost = gl.abs()[:, None] + (0 if gh is None else gh.abs()[:, None] * (lnp + w.H[:, None]))
        off = off + 2.0 ** -126 * scale * lost
        close(dx, want, (want.abs() + off) * U[t] + off + TINY[t], what)


@pytest.mark.parametrize("seed", SEEDS)
def test_random_clipping(seed):
    r, g = random.Random(300 + seed), torch.Generator().manual_seed(seed)
    n = r.choice([1, 3, 40, 56, 57, 130])
    host = [clip.rnd(g, (size(r, 200), size(r, 3000)), r.choice([BF, FP, F32]), r.choice([1e-3, 1.0]))
            for _ in range(n)]
    put = [clip.placed(t, r.choice(["plain", "off", "transposed", "rows"])) for t in host]
    want = clip.norm64(host)
    most, ws = clip.f32(want * r.choice([0.1, 0.7, 2.0])), Exact()
    c = min(1.0, most / want)
    if r.random() < 0.5:
        norm = d3.clip_grad_norm([v for v, _ in put], most, ws=ws)
        outs = [(v, b, c * t.double(), U[t.dtype] + (0 if t.dtype == F32 else 1.01 * EPS32), TINY[t.dtype])
                for t, (v, b) in zip(host, put)]
    else:
        sums = [clip.rnd(g, t.shape, F32) for t in host]
        to = []
        for (v, _), m in zip(put, sums):
            columns = not v.is_contiguous() and v.stride(1) != 1
            to.append(clip.placed(m, "transposed" if columns else r.choice(["plain", "off", "rows"])))
        norm = d3.clip_grad_norm([v for v, _ in put], most, into=[v for v, _ in to], ws=ws)
        outs = [(v, b, m.double() + c * t.double(), EPS32, 1e-45)
                for t, m, (v, b) in zip(host, sums, to)]
        assert all(torch.equal(v.cpu(), t) for t, (v, _) in zip(host, put)), seed
    ws.check(seed)
    assert abs(float(norm) - want) <= want * EPS32 * 1.001, seed
    for v, buf, w, rel, tiny in outs:
        close(v, w, w.abs() * rel * 1.0001 + tiny, (seed, v.shape))
        assert (clip.around(v, buf) == 7).all(), seed
