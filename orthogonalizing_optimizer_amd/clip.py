"""The global norm of many gradients, and their clipping.

Each function is one call of libdion3.so (include/dion3.h states the
formulas): two passes over the gradients, whatever their number, types and
shapes, without a copy to the host or to the device, so that they can be
captured into a graph.
"""
from __future__ import annotations

import array
from typing import Optional

import torch

from . import _lib
from .layer import _DTYPES, _call, _rows, _scratch, _size


def _whole(t) -> bool:
    """t's elements fill one stretch of memory, each once, in some order."""
    if t.is_contiguous():
        return True
    n = 1
    for stride, size in sorted((s, k) for k, s in zip(t.shape, t.stride()) if k != 1):
        if stride != n:
            return False
        n *= size
    return True


def _layout(g, m, i):
    """(rows, cols, row stride of g, row stride of m)."""
    n = g.numel()
    if m is None:
        if _whole(g):
            return 1, n, n, n
        rows, cols, ld = _rows(g, f"gradient {i}")
        return rows, cols, ld, cols
    if g.is_contiguous() and m.is_contiguous() or g.stride() == m.stride() and _whole(g):
        return 1, n, n, n
    rows, cols, ldg = _rows(g, f"gradient {i}")
    _, _, ldm = _rows(m, f"sum {i}")
    return rows, cols, ldg, ldm


def _plain(grads, into):
    """The table of contiguous tensors with elements, and the device; None
    where any is something else (then _table says what).  A pass over all
    tensors for each of their properties is cheaper than all checks a tensor
    (300 gradients into sums: 237 us, 314)."""
    try:
        device, index = grads[0].device, grads[0].get_device()
        if index < 0 or any([g.get_device() != index or g.requires_grad for g in grads]):
            return None
        if not all([g.is_contiguous() for g in grads]):
            return None
        codes = [_DTYPES[g.dtype] for g in grads]
        at, sizes = [g.data_ptr() for g in grads], [g.numel() for g in grads]
        if into is not None:
            if not all([m.dtype is torch.float32 and m.get_device() == index and m.is_contiguous()
                        and m.shape == g.shape for g, m in zip(grads, into)]):
                return None
            sums = [m.data_ptr() for m in into]
    except (AttributeError, KeyError, RuntimeError, IndexError, TypeError):
        return None
    if 0 in at or 0 in sizes:
        return None
    table = array.array("q", bytes(56 * len(grads)))
    table[0::7] = array.array("q", at)
    if into is not None:
        table[1::7] = array.array("q", sums)
    table[2::7] = array.array("q", [1]) * len(grads)
    table[3::7] = table[4::7] = table[5::7] = array.array("q", sizes)
    table[6::7] = array.array("q", codes)
    return table, device


def _table(grads, into, written):
    """(the library's table, its length, the device)."""
    grads = list(grads)
    if into is not None:
        into = list(into)
        if len(into) != len(grads):
            raise ValueError("need one sum per gradient")
    plain = _plain(grads, into)
    if plain is None:
        table, device = _checked(grads, into)
    else:
        table, device = plain
    if written:
        at = [m or g for m, g, n in zip(table[1::7], table[0::7], table[3::7]) if n]
        seen = set(at)
        if len(seen) != len(at):
            raise ValueError("a gradient or a sum is listed twice")
        if into is not None and not seen.isdisjoint(table[0::7]):
            raise ValueError("a sum is one of the gradients")
    return table, len(grads), device


def _checked(grads, into):
    """The table of tensors of any layout, and the device."""
    table, device = [], None
    strided, none = torch.strided, (0,) * 7
    for i, g in enumerate(grads):
        if g is None:
            table += none
            continue
        if not isinstance(g, torch.Tensor) or not g.is_cuda or g.layout is not strided:
            raise TypeError(f"gradient {i} must be a dense CUDA (HIP) tensor")
        if g.requires_grad:
            raise TypeError(f"gradient {i} requires a gradient itself: pass p.grad, not p")
        code = _DTYPES.get(g.dtype)
        if code is None:
            raise TypeError(f"gradient {i} must be float32, bfloat16 or float16")
        if device is None:
            device = g.device
        elif g.device != device:
            raise ValueError("all gradients must be on one device")
        m = None
        if into is not None:
            m = into[i]
            if not isinstance(m, torch.Tensor) or m.device != device or m.dtype is not torch.float32:
                raise TypeError(f"sum {i} must be a float32 tensor on {device}")
            if m.shape != g.shape:
                raise ValueError(f"sum {i} must have shape {tuple(g.shape)}")
        n = g.numel()
        if n == 0:
            table += none
            continue
        gp, mp = g.data_ptr(), 0 if m is None else m.data_ptr()
        if g.is_contiguous() and (m is None or m.is_contiguous()):
            table += (gp, mp, 1, n, n, n, code)
        else:
            table += (gp, mp, *_layout(g, m, i), code)
    return array.array("q", table), device


def grad_norm(grads, scale: float = 1.0, per_tensor: bool = False,
              ws: Optional[_lib.Workspace] = None):
    """scale * the square root of the sum of all the tensors' squares (0-dim
    fp32, on their device; squares are summed in 64 bits).  ``grads``: tensors
    of one device, fp32, bf16 or fp16; None stands for no gradient.  With
    ``per_tensor`` (norm, norms): norms[i] is the norm of tensor i alone."""
    table, count, device = _table(grads, None, False)
    if device is None:
        norm = torch.zeros(())
        return (norm, torch.zeros(count)) if per_tensor else norm
    at = table.buffer_info()[0]
    norm = torch.empty((), dtype=torch.float32, device=device)
    norms = torch.empty(count, dtype=torch.float32, device=device) if per_tensor else None
    p, nb, keep = _scratch(ws, _size("dion3_grad_norm_workspace_size", at, count), device)
    _call("dion3_grad_norm", device, at, count, float(scale), norm.data_ptr(),
          norms.data_ptr() if per_tensor else None, p, nb)
    return (norm, norms) if per_tensor else norm


def clip_grad_norm(grads, max_norm: float, scale: float = 1.0, into=None,
                   ws: Optional[_lib.Workspace] = None):
    """Scale the gradients in place by ``scale`` * min(1, max_norm / norm), with
    norm = ``grad_norm(grads, scale)``, and return norm.  ``scale``: 1 / the
    loss's scale, for fp16.  A norm that is infinite zeroes the finite
    gradients, one that is NaN makes all of them NaN.

    ``into``: fp32 tensors, one for each gradient and of its shape; the scaled
    gradients are then added to them and the gradients stay as they are.  For
    the momenta of a ``Dion3`` use its ``accumulate_clipped``, which steps the
    parameters that have a gradient here and no others.

    No tensor that is written may be listed twice or overlap another one.
    Pass gradients, not parameters; None stands for no gradient."""
    table, count, device = _table(grads, into, True)
    if device is None:
        return torch.zeros(())
    at = table.buffer_info()[0]
    norm = torch.empty((), dtype=torch.float32, device=device)
    p, nb, keep = _scratch(ws, _size("dion3_grad_norm_workspace_size", at, count), device)
    _call("dion3_clip_grad_norm", device, at, count, float(max_norm), float(scale),
          norm.data_ptr(), p, nb)
    return norm
