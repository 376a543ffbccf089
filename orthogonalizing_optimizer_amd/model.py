"""Operators around the layers in a model's training step.

Tokens' rows of an embedding (``embedding``); queries and keys normed per head
and rotated by their positions in one pass (``qk_norm_rope``); log
probabilities of given tokens with the entropy and the best alternatives
(``log_probs``); their gradients.  As in ``layer``, every function is one call
of libdion3.so (include/dion3.h states the formulas), runs on torch's current
stream of the tensors' device and takes its workspace from torch's allocator
per call (or from ``ws``); there is no fallback.

``embedding_layer``, ``qk_norm_rope_layer`` and ``token_log_probs`` are the
differentiable forms.  torch's rule for a captured backward pass holds: let no
graph of the same leaves recorded outside the capture live (an earlier loss or
output kept in a variable).
"""
from __future__ import annotations

import array
import functools
from typing import Optional

import torch

from . import _lib
from .layer import _DTYPES, _as_rows, _call, _matrix, _ptr, _rows, _same, _scratch, _size, _t16, _vector

_MAX_STRIDE = 1 << 38
# (these depend on sizes alone; a call to ask for one takes 1.4 us)
_bytes = functools.lru_cache(maxsize=1024)(_size)


def _lead(shape, strides, name):
    """(entries, the one stride of the leading dimensions) of a tensor of that
    shape and strides, None as the stride of a single entry."""
    n, ld = 1, None
    for size, stride in zip(reversed(shape), reversed(strides)):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif size > 0 and n > 0 and stride != ld * n:
            raise ValueError(f"{name}: its leading dimensions do not share one stride")
        n *= size
    return n, ld


# ----------------------------------------------------------- embedding

def _indices(t, shape, device, name):
    """(t contiguous, its bits): whole numbers, one a token."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError(f"{name} must be a tensor on {device}")
    if t.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"{name} must be int64 or int32")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.contiguous(), 64 if t.dtype == torch.int64 else 32


def embedding(tokens, w, scale: float = 1.0, dtype=None):
    """scale * w[tokens], rounded once to ``dtype``: [..., m] for tokens [...]
    (int64 or int32) and w [n, m].  ``dtype`` is w's type (the default) or, for
    fp32 w, also bf16 or fp16.  A token outside [0, n) stands for none: its row
    is zeros."""
    if not isinstance(w, torch.Tensor) or w.device.type != "cuda":
        raise TypeError("w must be a CUDA (HIP) tensor")
    dtype = w.dtype if dtype is None else dtype
    if w.dtype not in _DTYPES or dtype not in _DTYPES or w.dtype not in (torch.float32, dtype):
        raise TypeError("w must be float32 or of dtype, dtype float32, bfloat16 or float16")
    n, m, ldw = _matrix(w, w, "w")
    if not isinstance(tokens, torch.Tensor):
        raise TypeError(f"tokens must be a tensor on {w.device}")
    tokens, bits = _indices(tokens, tokens.shape, w.device, "tokens")
    y = w.new_empty(tokens.shape + (m,), dtype=dtype)
    _call("dion3_embedding", w.device, _ptr(tokens), bits, _ptr(w), ldw, _DTYPES[w.dtype], _ptr(y), m,
          tokens.numel(), n, m, float(scale), _DTYPES[dtype])
    return y


def embedding_grad(tokens, dy, n: int, scale: float = 1.0, out=None, accumulate: bool = False,
                   ws: Optional[_lib.Workspace] = None):
    """The gradient of ``embedding`` in its n rows, fp32: row v is scale times
    the sum of the rows of dy whose token is v (the same bits for the same
    tokens and dy).  With ``out`` (fp32 [n, m], contiguous rows) it is written
    there, and with ``accumulate`` added to it (a tied head's gradient, say):
    rows without tokens are then left alone."""
    if not isinstance(dy, torch.Tensor) or dy.device.type != "cuda":
        raise TypeError("dy must be a CUDA (HIP) tensor")
    if dy.dtype not in _DTYPES:
        raise TypeError("dy must be bfloat16, float16 or float32")
    T, m, lddy = _rows(dy, "dy")
    tokens, bits = _indices(tokens, dy.shape[:-1], dy.device, "tokens")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = dy.new_empty((n, m), dtype=torch.float32)
    if not isinstance(out, torch.Tensor) or out.device != dy.device or out.dtype != torch.float32:
        raise TypeError(f"out must be a float32 tensor on {dy.device}")
    if tuple(out.shape) != (n, m):
        raise ValueError(f"out must have shape {(n, m)}")
    _, _, ldw = _rows(out, "out")
    p, nb, keep = _scratch(ws, _bytes("dion3_embedding_grad_workspace_size", T, n, m), dy.device)
    _call("dion3_embedding_grad", dy.device, _ptr(tokens), bits, _ptr(dy), lddy, _ptr(out), ldw,
          int(bool(accumulate)), T, n, m, float(scale), _DTYPES[dy.dtype], p, nb)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, w, tokens, scale, dtype):
        ctx.save_for_backward(tokens)
        ctx.scale, ctx.n, ctx.wtype = scale, w.shape[0], w.dtype
        return embedding(tokens, w, scale, dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        tokens, = ctx.saved_tensors
        dw = embedding_grad(tokens, _as_rows(dy), ctx.n, ctx.scale)
        return dw.to(ctx.wtype), None, None, None


def embedding_layer(tokens, w, scale: float = 1.0, dtype=None):
    """``embedding``, differentiable in w (a dense gradient of w's type, summed
    in fp32)."""
    return _Embedding.apply(w, tokens, float(scale), dtype)


# ------------------------------------------------- heads: norm and rotation

def _heads(t, name):
    """(tokens, token stride, heads, head stride, columns) of [..., heads, columns]."""
    shape = t.shape
    if len(shape) < 2:
        raise ValueError(f"{name} must be [..., heads, columns]")
    h, D = shape[-2:]
    if h < 1 or D < 1:
        raise ValueError(f"{name} needs at least one head and one column")
    if t.is_contiguous():
        return t.numel() // (h * D), h * D, h, D, D
    strides = t.stride()
    if D > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must have contiguous columns")
    T, ld = _lead(shape[:-2], strides[:-2], name)
    hs = strides[-2] if h > 1 else D
    ld = h * D if ld is None else ld
    if (T > 1 and ld < D) or hs < D:
        raise ValueError(f"{name}: its heads overlap")
    return T, ld, h, hs, D


def _positions(positions, lead, device):
    if not isinstance(positions, torch.Tensor) or positions.device != device:
        raise TypeError(f"positions must be a tensor on {device}")
    if positions.dtype is not torch.int64 and positions.dtype is not torch.int32:
        raise TypeError("positions must be int64 or int32")
    if positions.shape != lead:
        positions = positions.expand(lead)           # (torch's own error where it does not)
    return positions if positions.is_contiguous() else positions.contiguous()


def _freqs(freqs, D, device):
    if not isinstance(freqs, torch.Tensor) or freqs.device != device:
        raise TypeError(f"freqs must be a tensor on {device}")
    if freqs.dtype != torch.float64:
        raise TypeError("freqs must be float64")
    if freqs.dim() != 1 or 2 * freqs.shape[0] > D or not freqs.is_contiguous():
        raise ValueError(f"freqs must be a contiguous vector of at most {D // 2} entries")
    return 2 * freqs.shape[0]


class _Sides:
    """The checked queries and keys of a call, as the library takes them: a
    dion3_heads each (its members in order, all of 8 bytes)."""

    __slots__ = ("q", "k", "T", "D", "r", "pos", "bits", "desc", "wtype", "dtype", "keep")

    def __init__(self, q, k, q_weight, k_weight, positions, freqs):
        _t16(q, "q")
        self.q, self.k = q, k
        self.T, ld, hq, hs, D = _heads(q, "q")
        self.D = D
        lead = q.shape[:-2]
        _vector(q_weight, D, q, "q_weight")
        # X, ldx, hsx, w, dY, lddy, hsdy, Y, ldy, hsy, heads
        self.desc = [[q.data_ptr(), ld, hs, q_weight.data_ptr(), 0, 0, 0, 0, 0, 0, hq], None]
        if (k is None) != (k_weight is None):
            raise ValueError("k and k_weight belong together")
        if k is not None:
            _same(k, q, "k")
            _, ld, hk, hs, Dk = _heads(k, "k")
            if k.shape[:-2] != lead or Dk != D:
                raise ValueError(f"k must have q's tokens and {D} columns a head")
            _vector(k_weight, D, q, "k_weight")
            if k_weight.dtype != q_weight.dtype:
                raise TypeError("q_weight and k_weight must have one type")
            self.desc[1] = [k.data_ptr(), ld, hs, k_weight.data_ptr(), 0, 0, 0, 0, 0, 0, hk]
        self.pos = _positions(positions, lead, q.device)
        self.r = _freqs(freqs, D, q.device)
        self.wtype, self.dtype = _DTYPES[q_weight.dtype], _DTYPES[q.dtype]
        self.bits = 64 if self.pos.dtype is torch.int64 else 32

    def output(self, i):
        """A contiguous output of side i, put into its description."""
        t = self.k if i else self.q
        y = t.new_empty(t.shape)
        d = self.desc[i]
        d[7], d[8], d[9] = y.data_ptr(), d[10] * self.D, self.D
        return y

    def refs(self):
        q, k = self.desc
        self.keep = a = array.array("q", q if k is None else q + k)
        p = a.buffer_info()[0]
        return p, None if k is None else p + 88


def qk_norm_rope(q, k, q_weight, k_weight, positions, freqs, eps: float = 1e-6,
                 interleaved: bool = False):
    """(yq, yk): queries [..., hq, D] and keys [..., hk, D] with each head
    normed, u = x / sqrt(mean x^2 + eps) * weight, and its first
    2 * len(freqs) columns turned by the angles positions * freqs: the pairs
    are columns (i, i + len(freqs)), or neighbours with ``interleaved``.

    q and k are bf16 or fp16 with contiguous columns and any strides of heads
    and tokens (views of one product's output, say; leading dimensions share a
    stride); outputs are contiguous.  Weights [D] are fp32 or of q's type.
    ``positions``: int64 or int32, one a token (or of a shape that expands to
    the tokens', which is copied to one a token).  ``freqs``: float64, radians a
    position, for instance base ** (-torch.arange(0, r, 2, dtype=torch.float64)
    / r).  k and k_weight may be None (queries alone; yk is None)."""
    s = _Sides(q, k, q_weight, k_weight, positions, freqs)
    yq = s.output(0)
    yk = s.output(1) if k is not None else None
    _call("dion3_qk_norm_rope", q.device, *s.refs(), _ptr(freqs), _ptr(s.pos), s.bits, s.T, s.D,
          s.r, int(bool(interleaved)), float(eps), s.wtype, s.dtype)
    return yq, yk


def qk_norm_rope_grad(dyq, dyk, q, k, q_weight, k_weight, positions, freqs, eps: float = 1e-6,
                      interleaved: bool = False, need_dx: bool = True, need_dw: bool = True,
                      ws: Optional[_lib.Workspace] = None):
    """(dq, dk, dq_weight, dk_weight) of ``qk_norm_rope`` from its inputs; the
    weights' gradients are fp32.  What is not needed comes back as None."""
    s = _Sides(q, k, q_weight, k_weight, positions, freqs)
    if (dyk is None) != (k is None):
        raise ValueError("k and its gradient belong together")
    for i, (dy, t) in enumerate(((dyq, q), (dyk, k))):
        if t is not None:
            _same(dy, t, "dyq" if i == 0 else "dyk", t.shape)
            _, ld, _, hs, _ = _heads(dy, "dyq" if i == 0 else "dyk")
            s.desc[i][4:7] = dy.data_ptr(), ld, hs
    if not need_dx and not need_dw:
        return None, None, None, None
    dq = s.output(0) if need_dx else None
    dk = s.output(1) if need_dx and k is not None else None
    dw = q.new_empty((2, s.D), dtype=torch.float32) if need_dw else None
    p, nb, keep = _scratch(ws, _bytes("dion3_qk_norm_rope_grad_workspace_size", s.T, q.shape[-2],
                                      k.shape[-2] if k is not None else 0, s.D, s.r,
                                      int(bool(interleaved))) if need_dw else 0, q.device)
    _call("dion3_qk_norm_rope_grad", q.device, *s.refs(), _ptr(freqs), _ptr(s.pos), s.bits, _ptr(dw),
          s.T, s.D, s.r, int(bool(interleaved)), float(eps), s.wtype, s.dtype, p, nb)
    return (dq, dk, dw[0] if need_dw else None,
            dw[1] if need_dw and k is not None else None)


def _as_heads(t):
    """A gradient as its producer left it, or contiguous where the library does
    not read its layout: that is autograd's choice, not the user's."""
    try:
        _, ld, _, hs, _ = _heads(t, "gradient")
        if max(ld, hs) <= _MAX_STRIDE:
            return t
    except ValueError:
        pass
    return t.contiguous()


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, freqs, eps, interleaved):
        yq, yk = qk_norm_rope(q, k, q_weight, k_weight, positions, freqs, eps, interleaved)
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, freqs)
        ctx.set_materialize_grads(False)
        ctx.eps, ctx.interleaved = eps, interleaved
        return yq, yk

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, positions, freqs = ctx.saved_tensors
        out = [None] * 8
        # the sides that a gradient reaches, and of these what is asked for
        sides = [(i, dy, x, w) for i, (dy, x, w) in enumerate(((dyq, q, wq), (dyk, k, wk)))
                 if dy is not None and (ctx.needs_input_grad[i] or ctx.needs_input_grad[2 + i])]
        if not sides:
            return tuple(out)
        args = [(_as_heads(dy), x, w) for _, dy, x, w in sides] + [(None, None, None)]
        (dy0, x0, w0), (dy1, x1, w1) = args[:2]
        need_dx = any(ctx.needs_input_grad[i] for i, *_ in sides)
        need_dw = any(ctx.needs_input_grad[2 + i] for i, *_ in sides)
        dx0, dx1, dw0, dw1 = qk_norm_rope_grad(dy0, dy1, x0, x1, w0, w1, positions, freqs, ctx.eps,
                                               ctx.interleaved, need_dx, need_dw)
        for (i, _, _, w), dx, dw in zip(sides, (dx0, dx1), (dw0, dw1)):
            if ctx.needs_input_grad[i]:
                out[i] = dx
            if ctx.needs_input_grad[2 + i]:
                out[2 + i] = dw.to(w.dtype)
        return tuple(out)


def qk_norm_rope_layer(q, k, q_weight, k_weight, positions, freqs, eps: float = 1e-6,
                       interleaved: bool = False):
    """``qk_norm_rope``, differentiable in q, k and the weights.  Kept for the
    backward pass: q and k as they are."""
    return _QkNormRope.apply(q, k, q_weight, k_weight, positions, freqs, float(eps),
                             bool(interleaved))


# ------------------------------------------------------ log probabilities

def _logits(x):
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise TypeError("logits must be a CUDA (HIP) tensor")
    if x.dtype not in _DTYPES:
        raise TypeError("logits must be bfloat16, float16 or float32")
    return _rows(x, "logits")


def _per_row(t, shape, device, name):
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.float32:
        raise TypeError(f"{name} must be a float32 tensor on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.contiguous()


def log_probs(logits, targets=None, scale: float = 1.0, entropy: bool = False, top: int = 0,
              ws: Optional[_lib.Workspace] = None):
    """(logp, stats, entropy, top_logp, top_index) of rows of logits [..., n]
    (bf16, fp16 or fp32) times ``scale`` (one over a temperature), all fp32 but
    the int64 indices; what is not asked for is None.

    ``targets`` [...] (int64 or int32): logp is their log probability; one
    outside [0, n) (a padded place's -100) gets 0.  stats [..., 2] holds the
    maximum m and l = ln sum exp(z - m): their sum is the log of the sum of
    exponentials, and ``log_probs_grad`` reads them.  A finite logit whose
    product with ``scale`` passes fp32's lowest number counts as that number:
    only a row of -infinity has no probabilities.  ``top`` (up to 64): the
    best alternatives' log probabilities and indices [..., top], best first,
    equal logits by their index."""
    T, n, ld = _logits(logits)
    lead, device = logits.shape[:-1], logits.device
    bits = 0
    logp = H = tl = ti = None
    if targets is not None:
        targets, bits = _indices(targets, lead, device, "targets")
        logp = logits.new_empty(lead, dtype=torch.float32)
    stats = logits.new_empty(lead + (2,), dtype=torch.float32)
    if entropy:
        H = logits.new_empty(lead, dtype=torch.float32)
    if top:
        if not 0 < top <= n:
            raise ValueError(f"top must be between 0 and {n}")
        tl = logits.new_empty(lead + (top,), dtype=torch.float32)
        ti = logits.new_empty(lead + (top,), dtype=torch.int64)
    p, nb, keep = _scratch(ws, _bytes("dion3_log_probs_workspace_size", T, n, top), device)
    _call("dion3_log_probs", device, _ptr(logits), ld, _ptr(targets), bits, _ptr(logp), _ptr(stats),
          _ptr(H), _ptr(tl), _ptr(ti), T, n, top, float(scale), _DTYPES[logits.dtype], p, nb)
    return logp, stats, H, tl, ti


def log_probs_grad(dlogp, logits, targets, stats, scale: float = 1.0, entropy=None, dentropy=None,
                   out=None):
    """The gradient in the logits, in their type, from the gradients of logp
    and (with ``entropy`` and ``dentropy``) of the entropy; ``dlogp`` and
    ``targets`` may both be None.  ``out``: where it is written, for instance
    over the logits themselves."""
    T, n, ld = _logits(logits)
    lead, device = logits.shape[:-1], logits.device
    if (dlogp is None) != (targets is None):
        raise ValueError("dlogp and targets belong together")
    if dlogp is None and dentropy is None:
        raise ValueError("need the gradient of logp, of the entropy or of both")
    bits = 0
    if targets is not None:
        targets, bits = _indices(targets, lead, device, "targets")
        dlogp = _per_row(dlogp, lead, device, "dlogp")
    stats = _per_row(stats, lead + (2,), device, "stats")
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs the entropy")
        entropy = _per_row(entropy, lead, device, "entropy")
        dentropy = _per_row(dentropy, lead, device, "dentropy")
    if out is None:
        out = logits.new_empty(logits.shape)
    _same(out, logits, "out", logits.shape)
    _, _, ldo = _rows(out, "out")
    _call("dion3_log_probs_grad", device, _ptr(dlogp), _ptr(logits), ld, _ptr(targets), bits,
          _ptr(stats), _ptr(entropy) if dentropy is not None else None, _ptr(dentropy), _ptr(out),
          ldo, T, n, float(scale), _DTYPES[logits.dtype])
    return out


class _TokenLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, scale, entropy):
        logp, stats, H, _, _ = log_probs(logits, targets, scale, entropy)
        ctx.save_for_backward(logits, targets, stats, H)
        ctx.set_materialize_grads(False)
        ctx.scale = scale
        return logp, H

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dlogp, dentropy):
        logits, targets, stats, H = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None, None
        if dlogp is None:
            targets = None
        return (log_probs_grad(dlogp, logits, targets, stats, ctx.scale, H, dentropy),
                None, None, None)


def token_log_probs(logits, targets, scale: float = 1.0, entropy: bool = False):
    """(logp, entropy) of ``log_probs``, differentiable in the logits; entropy
    is None unless asked for.  -logp.sum() / count is the cross entropy over
    the rows whose target is a token.  Kept for the backward pass: the logits
    and two or three fp32 values a row."""
    return _TokenLogProbs.apply(logits, targets, float(scale), bool(entropy))
