"""Shape-grouped Dion3 step over a set of weight matrices.

Transformers hold only a few distinct weight shapes; the matrices of one
shape are stepped together ("Dion3: Full-Stack Orthogonal Updates",
agihunt.info, level-4 paragraph: megabatching; here on one GPU, where it
turns one launch sequence per matrix into one per shape), and all shape
groups of a device go to the library in one call, which runs the s x s
products of groups with equal Gram sides as one launch.
"""
from __future__ import annotations

import math
from collections import OrderedDict
from fractions import Fraction
from typing import Dict, List, Optional, Sequence, Tuple

from . import _lib


class Dion3Step:
    """Holds (W, M) pairs, grouped by (shape, row stride).

    ``step()`` runs, per group, l1 row scoring, top-k selection with
    k = ceil(f n), Gram Newton-Schulz on the selected rows, the row-sparse
    update W[S] -= lr_eff * O with lr_eff = lr / sqrt(f) (level-3 paragraph:
    eta proportional to 1/sqrt(f)) and the decay M[S] *= mu.  The momentum M
    is the optimizer state.  ``step(grads)`` first accumulates one gradient
    per weight into it (M <- M + G, fused into the row scoring); ``step()``
    starts from M as it is.
    """

    def __init__(self, weights: Sequence, momenta: Sequence, lr: float = 0.02,
                 fraction=Fraction(1, 4), mu: float = 0.95, cfg: Optional[_lib.NsCfg] = None):
        if len(weights) != len(momenta):
            raise ValueError("need one momentum per weight")
        self.lr = float(lr)
        self.fraction = fraction
        self.mu = float(mu)
        self.cfg = cfg
        self.groups: "OrderedDict[Tuple, Dict]" = OrderedDict()
        self._order = list(weights)
        for w, m in zip(weights, momenta):
            if w.dim() != 2 or w.shape != m.shape:
                raise ValueError("Dion3 steps 2-D matrices with same-shape momentum")
            if w.stride() != m.stride() or w.stride(1) != 1 or w.device != m.device:
                raise ValueError("W and M must share strides and device, with contiguous rows")
            key = (tuple(w.shape), w.stride(0), str(w.device))
            self.groups.setdefault(key, {"W": [], "M": []})
            self.groups[key]["W"].append(w)
            self.groups[key]["M"].append(m)
        self.ws: Dict[str, _lib.Workspace] = {}     # one per device, shared by its groups
        for key, g in self.groups.items():
            dev = g["M"][0].device
            self.ws.setdefault(str(dev), _lib.Workspace())
            g["k"] = _lib.k_from_fraction(float(self.fraction), key[0][0])
            g["group"] = _lib.Group(g["W"], g["M"], g["k"], self.lr_eff)

    @property
    def lr_eff(self) -> float:
        return self.lr / math.sqrt(float(self.fraction))

    def step(self, grads: Optional[Sequence] = None):
        """One step over every group.  With ``grads`` (one per weight, in the
        order the weights were given), each momentum first accumulates its
        gradient, M <- M + G, fused into the row scoring."""
        gmap = None
        if grads is not None:
            if len(grads) != sum(len(g["W"]) for g in self.groups.values()):
                raise ValueError("need one gradient per weight")
            gmap = {id(w): gr for w, gr in zip(self._order, grads)}
        by_dev: "OrderedDict[str, List]" = OrderedDict()
        for key, g in self.groups.items():
            grp = g["group"]
            if gmap is not None:
                grp = _lib.Group(g["W"], g["M"], g["k"], self.lr_eff,
                                 Gs=[gmap[id(w)] for w in g["W"]])
            by_dev.setdefault(key[2], []).append(grp)
        for dev, grps in by_dev.items():
            for i in range(0, len(grps), _lib.MAX_GROUPS):
                _lib.step_groups(grps[i:i + _lib.MAX_GROUPS], self.mu, self.cfg, ws=self.ws[dev])


def _optimizer_base():
    import torch
    return torch.optim.Optimizer


def _stream(t):
    """The current stream of t's device; None for a host tensor."""
    import torch
    return torch.cuda.current_stream(t.device) if t.is_cuda else None


def _capturing(stream) -> bool:
    """Whether a graph is being captured from this stream."""
    import torch
    if stream == torch.cuda.current_stream():
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _follow(here, last):
    """Stream ``here`` waits for what ``last`` holds so far."""
    here.wait_stream(last)


def _hold(t, stream):
    """t's memory, made on another stream, is not given away while ``stream`` may use it."""
    t.record_stream(stream)


class Dion3(_optimizer_base()):
    """torch.optim-style Dion3 for 2-D fp32 parameters.

    Each parameter p with a gradient keeps a momentum buffer M (fp32, zero at
    first).  ``step()`` runs, per parameter group and per (shape, strides,
    device), one megabatched library call: M <- M + grad (fused into the row
    scoring), top-k row selection with k = ceil(f n), Gram Newton-Schulz on
    the selected rows, p[S] -= lr / sqrt(f) * O and M[S] *= mu ("Dion3:
    Full-Stack Orthogonal Updates", agihunt.info, level-3 paragraph: error
    feedback keeps the unselected rows of M for a later step; level-4:
    megabatching by shape).  Parameters that are not 2-D fp32 matrices with
    contiguous rows are refused: route them to another optimizer.

    With ``normalize=True`` the update is normalized per neuron (row) with a
    float32 second-moment state per row (``beta2``, ``eps``), the reading of
    the pages' "per-neuron normalization inherited from NorMuon" stated in
    include/dion3.h at dion3_norm_cfg.

    A layer may sum its weight gradient straight into the momentum
    (``linear_layer(..., into=optimizer)``): M <- M + dW where the product is
    computed, instead of a gradient buffer that ``step()`` adds.  The sums are
    the same.  Such a parameter has no ``.grad``; ``step()`` steps the ones
    that ``accumulate_grad`` has named since the last step.  A captured
    backward pass names none, neither when it is captured nor when it is
    replayed: for every parameter that it sums into, call
    ``accumulate_grad(p)`` before the replay, on the replay's stream.
    """

    def __init__(self, params, lr: float = 0.02, fraction=Fraction(1, 4), mu: float = 0.95,
                 cfg: Optional[_lib.NsCfg] = None, normalize: bool = False,
                 beta2: float = 0.95, eps: float = 1e-8):
        if lr <= 0 or not (0 < float(fraction) <= 1) or not (0 <= mu <= 1):
            raise ValueError("need lr > 0, 0 < fraction <= 1 and 0 <= mu <= 1")
        if normalize and not (0 <= beta2 < 1 and eps >= 0):
            raise ValueError("need 0 <= beta2 < 1 and eps >= 0")
        super().__init__(params, dict(lr=lr, fraction=fraction, mu=mu, normalize=normalize,
                                      beta2=beta2, eps=eps))
        import torch
        for group in self.param_groups:
            for p in group["params"]:
                if p.dim() != 2 or p.dtype != torch.float32 or p.stride(1) != 1:
                    raise ValueError("Dion3 steps 2-D fp32 matrices with contiguous rows")
        self.cfg = cfg
        self._ws: Dict[str, _lib.Workspace] = {}
        self._accumulated = set()      # parameters whose momentum already holds a new gradient
        # The stream that used a parameter's momentum last.  Sums into one
        # buffer read and write it without atomics, each on its layer's own
        # stream, and autograd, which sees none of them, does not order them:
        # a use on another stream waits for the last one.  Uses inside captures
        # are kept apart, since nothing there can wait for work outside.
        self._last: Dict = {}
        self._last_captured: Dict = {}

    def check_parameter(self, p):
        """Raise ValueError unless p is one of this optimizer's parameters, and
        RuntimeError where its momentum would be made inside a captured graph
        (every replay would clear it): call ``momentum(p)`` before."""
        if p not in self.state and not any(p is q for group in self.param_groups
                                           for q in group["params"]):
            raise ValueError("not a parameter of this optimizer")
        if p.is_cuda and "momentum" not in self.state.get(p, ()):
            import torch
            with torch.cuda.device(p.device):
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("a parameter's momentum must exist before the capture")

    def _buffer(self, p):
        """p's momentum buffer, made on the current stream if need be."""
        st = self.state[p]
        if "momentum" not in st:       # the parameter's own strides
            import torch
            st["momentum"] = torch.empty_strided(p.shape, p.stride(), dtype=p.dtype,
                                                 device=p.device).zero_()
            here = _stream(p)
            if here is not None:
                self._last[p] = here
        return st["momentum"]

    def _use(self, p):
        """(p's momentum buffer, whether the use is part of a capture), the
        current stream of its device behind the buffer's last use."""
        self.check_parameter(p)
        m = self._buffer(p)
        here = _stream(m)
        if here is None:
            return m, False
        captured = _capturing(here)
        uses = self._last_captured if captured else self._last
        last = uses.get(p)
        if last is not None and last != here and (not captured or _capturing(last)):
            _follow(here, last)
            if not captured:
                _hold(m, here)
        uses[p] = here
        return m, captured

    def momentum(self, p):
        """p's momentum buffer (fp32, p's strides; zero before the first
        gradient), to be used on the current stream of its device: that stream
        waits for the buffer's last use on another one, and the next use on
        another stream waits for this one."""
        return self._use(p)[0]

    def accumulate_grad(self, p):
        """p's momentum buffer (``momentum(p)``), for a gradient to be added to
        it on the current stream of its device: the next ``step()`` waits for
        that stream and steps p whether or not it has a ``.grad``.  Inside a
        capture nothing is added yet, and p is not named for the step."""
        m, captured = self._use(p)
        self._name(p, captured)
        return m

    def _name(self, p, captured):
        if not captured:
            self._accumulated.add(p)

    def load_state_dict(self, state_dict):
        """As in torch.  Gradients summed into a momentum since the last step
        are part of it: they go with the momentum that is replaced, and the
        next step does not count them.  A graph captured before sums into the
        momentum that was replaced: capture anew."""
        super().load_state_dict(state_dict)
        self._accumulated.clear()
        self._last.clear()
        for group in self.param_groups:
            for p in group["params"]:
                here = _stream(p)
                # (what is loaded was made there)
                if here is not None and "momentum" in self.state.get(p, ()):
                    self._last[p] = here

    @property
    def _streams(self):
        """Where the gradients that the next ``step()`` takes were added last."""
        return {self._last[p] for p in self._accumulated if p in self._last}

    def step(self, closure=None):
        import torch
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        # autograd runs a layer's backward on its forward's stream, and joins
        # that stream with the caller's only for gradients that it keeps itself
        params = [p for group in self.param_groups for p in group["params"]
                  if p.grad is not None or p in self._accumulated]
        here, followed = {}, set()
        for p in params:
            if p.device not in here:
                here[p.device] = _stream(p)
            stream, last = here[p.device], self._last.get(p)
            if last is None or last == stream:
                continue
            if last not in followed:
                followed.add(last)
                _follow(stream, last)
            _hold(self.state[p]["momentum"], stream)
        with torch.no_grad():
            for group in self.param_groups:
                f = float(group["fraction"])
                buckets: "OrderedDict[Tuple, List]" = OrderedDict()
                for p in group["params"]:
                    if p.grad is None and p not in self._accumulated:
                        continue
                    if p.grad is not None and p.grad.stride() != p.stride():
                        raise ValueError("a gradient must have its parameter's strides")
                    self._buffer(p)
                    st = self.state[p]
                    if group["normalize"] and "second_moment" not in st:
                        st["second_moment"] = torch.zeros(p.shape[0], dtype=torch.float32,
                                                          device=p.device)
                    buckets.setdefault((tuple(p.shape), p.stride(), str(p.device),
                                        p.grad is not None), []).append(p)
                # one library call per device over all of its shape buckets
                by_dev: "OrderedDict[str, List]" = OrderedDict()
                for (shape, _, dev, has_grad), ps in buckets.items():
                    k = _lib.k_from_fraction(f, shape[0])
                    Vs = ([self.state[p]["second_moment"] for p in ps] if group["normalize"]
                          else None)
                    by_dev.setdefault(dev, []).append(
                        _lib.Group(ps, [self.state[p]["momentum"] for p in ps], k,
                                   group["lr"] / math.sqrt(f),
                                   Gs=[p.grad for p in ps] if has_grad else None, Vs=Vs))
                norm = (group["beta2"], group["eps"]) if group["normalize"] else None
                for dev, grps in by_dev.items():
                    ws = self._ws.setdefault(dev, _lib.Workspace())
                    for i in range(0, len(grps), _lib.MAX_GROUPS):
                        _lib.step_groups(grps[i:i + _lib.MAX_GROUPS], group["mu"], self.cfg,
                                         norm=norm, ws=ws)
        for p in params:
            if here[p.device] is not None:
                self._last[p] = here[p.device]
        self._accumulated.clear()
        return loss
