"""Log probabilities of logits so large that their products with the scale are
rounded by more than an exponential holds: rows that a mask has filled with the
type's lowest value or with -1e30, at temperatures other than 1.

The formulas in 64 bits, with z = scale x held at fp32's lowest value where a
finite logit's product passes it.  A row's distances to its rounded maximum m are off by one residual
r = max z - m together (at most 32 below 2^30; above, products are rounded
first and r is 0), so the bounds below are those of the ordinary rows with
every distance moved by r."""
import math

import numpy as np
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests.layer_ref import EPS32, TINY, U, close, d

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
LOWEST = -float(np.finfo(np.float32).max)


class Far:
    """The formulas for rows x in 64 bits, and bounds."""

    def __init__(self, x, targets, scale):
        self.scale = float(np.float32(scale))
        z = d(x) * self.scale
        z = torch.where(torch.isinf(d(x)), z, z.clamp_min(LOWEST))
        self.top = z.amax(1, keepdim=True)
        self.m = self.top.float().double().clamp_min(LOWEST)
        r = torch.where(self.m.abs() < 2.0 ** 30, self.top - self.m, 0.0)
        dz = z - self.top
        l = torch.logsumexp(dz, 1, keepdim=True)
        self.q = dz - l
        self.p = torch.exp(self.q)
        near = torch.where(self.p > 0, dz + r, 0.0)                # distances as they are summed
        e1, e2 = (self.p * near.abs()).sum(1), (self.p * near * near).sum(1)
        lr = (l + r)[:, 0].abs()
        self.H = -torch.where(self.p > 0, self.p * self.q, 0.0).sum(1)
        self.lse = (self.top + l)[:, 0]
        s_off = (6 * e1 + 70) * EPS32
        self.l_off = s_off + (3 * lr + 2) * EPS32
        self.H_off = self.l_off + (6 * e2 + 74 * e1 + 2 * self.H + lr) * EPS32 + e1 * s_off
        self.j = targets
        self.logp = self.q.gather(1, targets[:, None])[:, 0]
        self.dz, self.r, self.l = dz, r, l
        self.logp_off = self.l_off + ((dz + r).gather(1, targets[:, None])[:, 0].abs()
                                      + self.logp.abs()) * EPS32

    def grad(self, g, gh):
        hot = torch.nn.functional.one_hot(self.j, self.q.shape[1]).double()
        g, gh = d(g)[:, None], d(gh)[:, None]
        lnp = torch.where(self.p > 0, self.q, 0.0)
        w = g * (hot - self.p) - gh * self.p * (lnp + self.H[:, None])
        size = g.abs() * self.p + gh.abs() * self.p * (lnp.abs() + self.H[:, None])
        off = ((4 * (lnp.abs() + (self.dz + self.r).abs().clamp_max(300) + self.r.abs()) + 24) * EPS32
               + self.l_off[:, None])
        # (a probability below 2^-126 may count as none)
        lost = 2.0 ** -126 * (g.abs() + gh.abs() * (110 + self.H[:, None]))
        return self.scale * w, self.scale * (size * off + gh.abs() * self.p * (self.H_off[:, None] + off)
                                             + g.abs() * hot * 4 * EPS32 + lost)


def check(x, targets, scale, what=""):
    w = Far(x, targets, scale)
    n = x.shape[1]
    t = targets.cuda()
    for top in (0, min(n, 2)):
        logp, stats, H, tl, ti = d3.log_probs(x.cuda(), t, scale=scale, entropy=True, top=top)
        assert torch.equal(d(stats[:, 0]), w.m[:, 0]), what
        close(H, w.H, w.H_off, (what, "entropy"))
        gone = torch.isinf(w.logp)
        assert (logp.cpu()[gone] == -math.inf).all(), what
        close(logp[~gone.cuda()], w.logp[~gone], w.logp_off[~gone], (what, "logp"))
        lse = d(stats).sum(1)
        close(lse, w.lse, w.l_off + 2 * w.lse.abs() * 2.0 ** -53
              + torch.where(w.m.abs() < 2.0 ** 30, 0.0, w.m.abs() * EPS32)[:, 0], (what, "lse"))
        if top:
            at = torch.sort(d(x), dim=1, descending=True, stable=True)[1][:, :top]
            assert torch.equal(ti.cpu(), at), what
            want, off = w.q.gather(1, at), (w.dz + w.r).gather(1, at).abs()
            low = torch.isinf(want)
            assert (tl.cpu()[low] == -math.inf).all(), what
            err = (d(tl) - want).abs()
            assert (err[~low] <= (w.l_off[:, None] + (off + want.abs()) * EPS32)[~low]).all(), what
    g = torch.Generator().manual_seed(n)
    gl, gh = torch.randn(len(x), generator=g), torch.randn(len(x), generator=g)
    for h in (torch.zeros_like(gh), gh):
        dx = d3.log_probs_grad(gl.cuda(), x.cuda(), t, stats, scale=scale, entropy=H,
                               dentropy=h.cuda() if h.any() else None)
        want, off = w.grad(gl, h)
        close(dx, want, (want.abs() + off) * U[x.dtype] + off + TINY[x.dtype], (what, "dx"))


FILLS = {BF: ["lowest", -1e30, -1e20, -1e10, 1e10, 1e30], FP: ["lowest", -3e4, 3e4],
         F32: ["lowest", -1e30, -1e20, -1e10, 1e10, 1e30]}


@pytest.mark.parametrize("scale", [1.0, 0.7, 0.9, 1.25, 3.1])
@pytest.mark.parametrize("n", [3, 100, 9000, 140000])
@pytest.mark.parametrize("dtype,fill", [(t, f) for t in FILLS for f in FILLS[t]])
def test_filled_rows(dtype, fill, n, scale):
    """All filled: 1 / n each.  Some -infinity: none there.  One ordinary logit
    among low ones, at either end: all of it.  Half of the row at half the
    value: the larger half."""
    low = torch.finfo(dtype).min if fill == "lowest" else fill
    x = torch.full((5, n), low, dtype=dtype)
    x[1, n // 2:] = -math.inf
    if low < 0:
        x[2, 0], x[3, n - 1] = 0.5, -2.5
    x[4, n // 2:] = low / 2
    check(x, torch.tensor([n - 1, 0, 0, n - 1, n - 1 if low < 0 else 0]), scale, (dtype, fill, n, scale))


def test_infinite_rows_stay_so():
    """Only rows of -infinity have no probability, whatever the scale."""
    x = torch.full((3, 50), -math.inf)
    x[1] = LOWEST
    x[2, 7] = LOWEST
    t = torch.tensor([7, 7, 7]).cuda()
    for scale in (0.7, 1.0, 1.25, 1e10):
        logp, stats, H, _, _ = d3.log_probs(x.cuda(), t, scale=scale, entropy=True)
        assert stats[0].tolist() == [-math.inf, 0.0] and logp[0] == -math.inf and H[0] == 0
        assert torch.isfinite(stats[1:]).all()
        assert abs(float(logp[1]) + math.log(50)) < 1e-5 and abs(float(H[1]) - math.log(50)) < 1e-5
        assert float(logp[2]) == 0 and float(H[2]) == 0


@pytest.mark.parametrize("scale", [0.7, 0.9, 1.3])
@pytest.mark.parametrize("base", [1e3, -3e4, 1e6, -1e7])
def test_logits_around_a_large_value(base, scale):
    """fp32 logits that differ by ordinary amounts."""
    g = torch.Generator().manual_seed(int(abs(base)))
    x = (base + 3 * torch.randn(6, 20000, generator=g, dtype=torch.float64)).float()
    check(x, torch.randint(0, 20000, (6,), generator=g), scale, (base, scale))
