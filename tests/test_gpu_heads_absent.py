"""Sums over heads and tokens where a batch of them is not full and eps is 0: a
slot without a head counts nothing (its statistic, 1 / sqrt(0), is infinite)."""
import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from tests import test_gpu_heads as heads
from tests.layer_ref import EPS32, close, d, rounded

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
# T, query heads, key heads, columns, turned columns: 5 and 12 heads of 8 a batch, tokens that do
# not fill a batch of several, ragged, lapped and whole pieces
SIZES = [(3, 5, 12, 128, 128), (7, 4, 1, 128, 128), (5, 12, 4, 128, 64), (9, 3, 1, 64, 64), (1, 1, 0, 16, 16),
         (5, 7, 2, 96, 24), (11, 5, 3, 80, 20), (3, 3, 2, 7, 4), (13, 2, 1, 33, 30), (2, 3, 1, 512, 512),
         (1001, 5, 1, 128, 128), (8191, 9, 1, 64, 32)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,hq,hk,D,r", SIZES)
def test_no_eps(T, hq, hk, D, r, dtype, interleaved):
    g = torch.Generator().manual_seed(T + D + r)
    q, k, wq, wk, fr = heads.inputs(g, T, hq, hk, D, r, dtype, torch.float32)
    q, k = (torch.where(x.abs() < 2.0 ** -7, 1.0, x).to(dtype) for x in (q, k))    # no head of zeros
    pos = torch.randint(0, 5000, (T,), generator=g)
    kc, wkc = (k.cuda(), wk.cuda()) if hk else (None, None)
    args = (q.cuda(), kc, wq.cuda(), wkc, pos.cuda(), fr.cuda())
    yq, yk = d3.qk_norm_rope(*args, eps=0.0, interleaved=interleaved)
    dyq, dyk = heads.rnd(g, T, hq, D, dtype=dtype), heads.rnd(g, T, max(hk, 1), D, dtype=dtype)
    dq, dk, dwq, dwk = d3.qk_norm_rope_grad(dyq.cuda(), dyk.cuda() if hk else None, *args, eps=0.0,
                                            interleaved=interleaved)
    for x, w, y, dy, dx, dw in ((q, wq, yq, dyq, dq, dwq), (k, wk, yk, dyk, dk, dwk))[:1 + (hk > 0)]:
        want, size = heads.formula(x, w, pos, fr, interleaved, 0.0)
        close(y, want, rounded(want, dtype, size * (heads.CHAIN / 2 + heads.TURN + 4) * EPS32), "y")
        wx, lim, ww, wl = heads.grad_formula(dy, x, w, pos, fr, interleaved, 0.0)
        close(dx, wx, rounded(wx, dtype, lim * (2 * heads.CHAIN + heads.TURN + 8) * EPS32), "dx")
        # 3072 waves share the batches, of which there are at most as many as heads; a
        # lane takes one head of each of its wave's; then 6 additions across lanes, 3
        # across waves, 12 of the workgroups' rows and 6 across their slices
        chain = T * (hq + hk) // 3072 + 2 + 6 + 3 + 12 + 6
        close(dw, ww, wl * (min(chain, T * x.shape[1]) + heads.CHAIN + heads.TURN) * EPS32 + 1e-30, "dw")


def test_layer_without_eps():
    g = torch.Generator().manual_seed(2)
    q, k, wq, wk, fr = heads.inputs(g, 3, 5, 1, 128, 128, BF, torch.float32)
    pos = torch.arange(3)
    qc, kc, a, b = (t.cuda().requires_grad_(True) for t in (q, k, wq, wk))
    yq, yk = d3.qk_norm_rope_layer(qc, kc, a, b, pos.cuda(), fr.cuda(), eps=0.0)
    (yq.float().sum() + yk.float().sum()).backward()
    for w, x, ws in ((a, q, wq), (b, k, wk)):
        _, _, ww, wl = heads.grad_formula(torch.ones_like(x), x, ws, pos, fr, False, 0.0)
        close(w.grad, ww, wl * (15 + heads.CHAIN + heads.TURN) * EPS32)
    assert torch.isfinite(d(qc.grad)).all() and torch.isfinite(d(kc.grad)).all()
