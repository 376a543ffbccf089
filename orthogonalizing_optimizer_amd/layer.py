"""Operators of the layers whose weights the optimizer steps.

The norm before a linear layer with the residual's addition
(``add_rms_norm``), the layer's product with bias, activation and residual in
its epilogue (``linear``), their gradients, and activations kept in 8 bits
between the forward and the backward pass (``pack_f8``, ``PackedF8``).  Every
function is one call of libdion3.so (include/dion3.h states the formulas);
nothing here computes, and there is no fallback.

Tensors are [..., features] on one GPU, bf16 or fp16, with contiguous
features; leading dimensions that share one stride (any row stride) are
flattened without a copy.  Calls run on torch's current stream of the
tensors' device.  Workspaces come from torch's allocator per call, so calls
on several streams or inside several captured graphs never share one; pass
``ws`` to manage the memory yourself.

``rms_norm_residual`` and ``linear_layer`` are the differentiable forms; the
latter can keep its inputs in 8 bits and sum its weight gradient straight
into the momentum of ``Dion3`` (see there).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib

F8_BLOCK = 32
_MAX_LD = 1 << 21                # the library's largest row stride
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


# ------------------------------------------------------------------ arguments

def _t16(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16")


def _same(t, like, name, shape=None):
    """t shares like's device and type (and has `shape`)."""
    if not isinstance(t, torch.Tensor) or t.device != like.device:
        raise TypeError(f"{name} must be a tensor on {like.device}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _vector(v, n, like, name):
    if not isinstance(v, torch.Tensor) or v.device != like.device:
        raise TypeError(f"{name} must be a tensor on {like.device}")
    if v.dtype not in (torch.float32, like.dtype):
        raise TypeError(f"{name} must be float32 or {like.dtype}")
    if v.dim() != 1 or v.shape[0] != n or (n > 1 and v.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} entries")


def _rows(t, name):
    """(rows, features, row stride) of a [..., features] tensor."""
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    m = t.shape[-1]
    if m < 1:
        raise ValueError(f"{name} needs at least one feature")
    if t.is_contiguous():
        return t.numel() // m, m, m
    if m > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous features")
    rows, ld = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif size > 0 and rows > 0 and stride != ld * rows:
            raise ValueError(f"{name}: its leading dimensions do not share one stride")
        rows *= size
    if rows <= 1:
        return rows, m, m
    if ld < m:
        raise ValueError(f"{name}: its rows overlap")
    return rows, m, ld


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _ptr(t):
    return None if t is None else t.data_ptr() or None     # (no tokens: no storage)


def _like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _scratch(ws, nbytes, device):
    """(pointer, bytes, what keeps it alive)."""
    if nbytes == 0:
        return None, 0, None
    if ws is not None:
        p, n = ws.get(nbytes, device)
        return p, n, ws
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    p = buf.data_ptr()
    return p + (-p) % 256, nbytes, buf


def _size(name, *args):
    out = ctypes.c_size_t(0)
    status = _fn(name)(*args, ctypes.byref(out))
    if status:
        _lib._check(status, name)
    return out.value


# The stream's handle without a torch.cuda.Stream around it (about 2 us a
# call, as much as a small kernel), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_fns: dict = {}                  # the library's entry points, looked up once


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(_lib.lib(), name)
    return f


def _call(name, device, *args):
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _lib._check(_fn(name)(*args, _lib._stream(device)), name)
    stream = _raw_stream(device.index) if _raw_stream is not None else _lib._stream(device)
    status = _fn(name)(*args, stream)
    if status:
        _lib._check(status, name)


# --------------------------------------------------------- the 8-bit format

class PackedF8:
    """An activation held in 8 bits: ``q`` (e4m3, [rows, cols rounded up to
    32]) and ``scale`` (uint8, one exponent byte per 32 columns of a row);
    a value is q * 2^(scale - 127).  ``shape`` is the shape of the tensor it
    stands for (default: [rows, cols])."""

    def __init__(self, q, scale, cols: int, shape=None):
        cp = -(-int(cols) // F8_BLOCK) * F8_BLOCK
        if not isinstance(q, torch.Tensor) or q.device.type != "cuda":
            raise TypeError("q must be a CUDA (HIP) tensor")
        if q.dtype != torch.float8_e4m3fn:
            raise TypeError("q must be float8_e4m3fn")
        if not isinstance(scale, torch.Tensor) or scale.device != q.device:
            raise TypeError(f"scale must be a tensor on {q.device}")
        if scale.dtype != torch.uint8:
            raise TypeError("scale must be uint8")
        if cols < 1 or q.dim() != 2 or q.shape[1] != cp or not q.is_contiguous():
            raise ValueError(f"q must be contiguous [rows, {cp}]")
        if tuple(scale.shape) != (q.shape[0], cp // F8_BLOCK) or not scale.is_contiguous():
            raise ValueError(f"scale must be contiguous [{q.shape[0]}, {cp // F8_BLOCK}]")
        if q.numel() and q.data_ptr() % 16:
            raise ValueError("q must be 16-byte aligned")
        self.q, self.scale, self.rows, self.cols = q, scale, q.shape[0], int(cols)
        self.shape = torch.Size(shape) if shape is not None else torch.Size((self.rows, self.cols))
        if self.shape[-1] != self.cols or self.shape.numel() != self.rows * self.cols:
            raise ValueError("shape does not hold these rows and columns")

    @property
    def device(self):
        return self.q.device

    @property
    def nbytes(self) -> int:
        return self.q.numel() + self.scale.numel()


def _empty_packed(like, rows, cols):
    """A PackedF8 to be filled, for `like`, whose rows and columns these are."""
    cp = -(-cols // F8_BLOCK) * F8_BLOCK
    p = PackedF8.__new__(PackedF8)
    p.q = like.new_empty((rows, cp), dtype=torch.float8_e4m3fn)
    p.scale = like.new_empty((rows, cp // F8_BLOCK), dtype=torch.uint8)
    p.rows, p.cols, p.shape = rows, cols, like.shape
    return p


def pack_f8(x) -> PackedF8:
    """x ([..., features], bf16, fp16 or fp32) in the 8-bit format."""
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise TypeError("x must be a CUDA (HIP) tensor")
    if x.dtype not in _DTYPES:
        raise TypeError("x must be bfloat16, float16 or float32")
    T, m, ld = _rows(x, "x")
    p = _empty_packed(x, T, m)
    _call("dion3_pack_f8", x.device, _ptr(x), ld, _ptr(p.q), _ptr(p.scale), T, m, _DTYPES[x.dtype])
    return p


def unpack_f8(p: PackedF8, dtype=torch.bfloat16):
    """The values that ``p`` stands for, in bf16, fp16 or fp32."""
    if not isinstance(p, PackedF8):
        raise TypeError("p must be a PackedF8")
    if dtype not in _DTYPES:
        raise TypeError("dtype must be bfloat16, float16 or float32")
    y = torch.empty(p.shape, dtype=dtype, device=p.device)
    _call("dion3_unpack_f8", p.device, _ptr(p.q), _ptr(p.scale), _ptr(y), p.cols, p.rows, p.cols,
          _DTYPES[dtype])
    return y


# ------------------------------------------------------------------- the norm

def add_rms_norm(x, weight, residual=None, eps: float = 1e-6, pack: bool = False,
                 return_y: bool = True):
    """(y, h, rstd, packed): h = x + residual rounded to x's type (x itself
    without a residual), rstd = 1 / sqrt(mean h^2 + eps) per row (fp32),
    y = h rstd weight, and with ``pack`` the 8-bit form of y.  ``weight`` is
    fp32 or of x's type.  ``return_y=False`` leaves y out (None)."""
    _t16(x, "x")
    T, m, ldx = _rows(x, "x")
    _vector(weight, m, x, "weight")
    h, ldr, ldh = x, 0, 0
    if residual is not None:
        _same(residual, x, "residual", x.shape)
        _, _, ldr = _rows(residual, "residual")
        h, ldh = _like(x), m
    if not return_y and not pack:
        raise ValueError("ask for y, its 8-bit form or both")
    y = _like(x) if return_y else None
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
    p = _empty_packed(x, T, m) if pack else None
    _call("dion3_add_rms_norm", x.device, _ptr(x), ldx, _ptr(residual), ldr, weight.data_ptr(),
          _DTYPES[weight.dtype], None if residual is None else _ptr(h), ldh, _ptr(y), m,
          _ptr(p.q) if p else None, _ptr(p.scale) if p else None, _ptr(rstd), T, m, float(eps),
          _DTYPES[x.dtype])
    return y, h, rstd, p


def add_rms_norm_grad(dy, h, rstd, weight, dh=None, need_dx: bool = True, need_dw: bool = True,
                      ws: Optional[_lib.Workspace] = None):
    """(dx, dweight) of ``add_rms_norm``: dx, the gradient of both x and the
    residual, includes ``dh``, the gradient that reaches h past the norm;
    dweight is fp32.  What is not needed comes back as None."""
    _t16(dy, "dy")
    T, m, ldy = _rows(dy, "dy")
    _same(h, dy, "h", dy.shape)
    _, _, ldh = _rows(h, "h")
    _vector(weight, m, dy, "weight")
    if (not isinstance(rstd, torch.Tensor) or rstd.device != dy.device
            or rstd.dtype != torch.float32):
        raise TypeError(f"rstd must be a float32 tensor on {dy.device}")
    if tuple(rstd.shape) != tuple(dy.shape[:-1]) or not rstd.is_contiguous():
        raise ValueError("rstd must be contiguous, one entry per row")
    lddh = 0
    if dh is not None:
        _same(dh, dy, "dh", dy.shape)
        _, _, lddh = _rows(dh, "dh")
    if not need_dx and not need_dw:
        return None, None
    dx = _like(dy) if need_dx else None
    dw = dy.new_empty(m, dtype=torch.float32) if need_dw else None
    p, nb, keep = _scratch(ws, _size("dion3_add_rms_norm_grad_workspace_size", T, m), dy.device)
    _call("dion3_add_rms_norm_grad", dy.device, _ptr(dy), ldy, _ptr(h), ldh, _ptr(rstd),
          weight.data_ptr(), _DTYPES[weight.dtype], _ptr(dh), lddh, _ptr(dx), m, _ptr(dw), T, m,
          _DTYPES[dy.dtype], p, nb)
    return dx, dw


# ------------------------------------------------------------ linear products

def _matrix(w, like, name):
    _same(w, like, name)
    if w.dim() != 2:
        raise ValueError(f"{name} must be [n, m]")
    n, m, ld = _rows(w, name)
    if n < 1:
        raise ValueError(f"{name} needs at least one row")
    return n, m, ld


def linear(x, w, bias=None, act: str = "none", residual=None, return_preact: bool = False,
           ws: Optional[_lib.Workspace] = None):
    """(y, z): z = x w^T + bias and y = act(z) + residual, with w [n, m] of
    x's type, ``bias`` fp32 or of x's type.  z comes back rounded with
    ``return_preact`` (for ``act_grad``), else as None."""
    _t16(x, "x")
    T, m, ldx = _rows(x, "x")
    n, wm, ldw = _matrix(w, x, "w")
    if wm != m:
        raise ValueError(f"w must have {m} columns")
    a = _act(act)
    shape = x.shape[:-1] + (n,)
    if bias is not None:
        _vector(bias, n, x, "bias")
    ldr = 0
    if residual is not None:
        _same(residual, x, "residual", shape)
        _, _, ldr = _rows(residual, "residual")
    y = x.new_empty(shape)
    z = x.new_empty(shape) if return_preact else None
    p, nb, keep = _scratch(ws, _size("dion3_linear_workspace_size", _ptr(x), ldx, w.data_ptr(), ldw,
                                     T, n, m), x.device)
    _call("dion3_linear", x.device, _ptr(x), ldx, w.data_ptr(), ldw, _ptr(bias),
          _DTYPES[bias.dtype] if bias is not None else 0, _ptr(residual), ldr, _ptr(y), n, _ptr(z),
          n, T, n, m, a, _DTYPES[x.dtype], p, nb)
    return y, z


def act_grad(dy, z, act: str, bias: bool = False, ws: Optional[_lib.Workspace] = None):
    """(dz, db): dz = dy act'(z) and with ``bias`` the sum of its rows (fp32,
    before rounding; else None).  z is the preactivation or its PackedF8, and
    may be None for "none", where dz is dy itself."""
    _t16(dy, "dy")
    T, n, ldy = _rows(dy, "dy")
    a = _act(act)
    zp = zq = zs = None
    ldz = 0
    if act != "none":
        if isinstance(z, PackedF8):
            if z.device != dy.device or tuple(z.shape) != tuple(dy.shape):
                raise ValueError(f"z must have shape {tuple(dy.shape)} on {dy.device}")
            zq, zs = _ptr(z.q), _ptr(z.scale)
        else:
            _same(z, dy, "z", dy.shape)
            _, _, ldz = _rows(z, "z")
            zp = _ptr(z)
    dz = _like(dy) if act != "none" else None
    db = dy.new_empty(n, dtype=torch.float32) if bias else None
    if dz is not None or db is not None:
        p, nb, keep = _scratch(ws, _size("dion3_act_grad_workspace_size", T, n) if bias else 0,
                               dy.device)
        _call("dion3_act_grad", dy.device, _ptr(dy), ldy, zp, ldz, zq, zs, _ptr(dz), n, _ptr(db), T,
              n, a, _DTYPES[dy.dtype], p, nb)
    return (dz if dz is not None else dy), db


def linear_grad_input(dz, w, residual=None, ws: Optional[_lib.Workspace] = None):
    """dx = dz w (+ residual, another branch's gradient of the same x)."""
    _t16(dz, "dz")
    T, n, lddz = _rows(dz, "dz")
    wn, m, ldw = _matrix(w, dz, "w")
    if wn != n:
        raise ValueError(f"w must have {n} rows")
    shape = dz.shape[:-1] + (m,)
    ldr = 0
    if residual is not None:
        _same(residual, dz, "residual", shape)
        _, _, ldr = _rows(residual, "residual")
    dx = dz.new_empty(shape)
    p, nb, keep = _scratch(ws, _size("dion3_linear_grad_input_workspace_size", _ptr(dz), lddz,
                                     w.data_ptr(), ldw, T, n, m), dz.device)
    _call("dion3_linear_grad_input", dz.device, _ptr(dz), lddz, w.data_ptr(), ldw, _ptr(residual),
          ldr, _ptr(dx), m, T, n, m, _DTYPES[dz.dtype], p, nb)
    return dx


def linear_grad_weight(dz, x, out=None, accumulate: bool = False,
                       ws: Optional[_lib.Workspace] = None):
    """dz^T x in fp32 ([n, m]); x is the layer's input or its PackedF8.  With
    ``out`` (fp32, contiguous rows) it is written there, and with
    ``accumulate`` added to it: ``out`` may be the optimizer's momentum."""
    _t16(dz, "dz")
    T, n, lddz = _rows(dz, "dz")
    lead = tuple(dz.shape[:-1])
    if isinstance(x, PackedF8):
        if x.device != dz.device:
            raise TypeError(f"x must be on {dz.device}")
        if x.rows != T or (tuple(x.shape[:-1]) != lead and len(lead) != 1):
            raise ValueError("x must have dz's rows")
        m, ldx, xp, sp = x.cols, x.cols, _ptr(x.q), _ptr(x.scale)
    else:
        _same(x, dz, "x")
        if tuple(x.shape[:-1]) != lead:
            raise ValueError("x must have dz's rows")
        _, m, ldx = _rows(x, "x")
        xp, sp = _ptr(x), None
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = dz.new_empty((n, m), dtype=torch.float32)
    if not isinstance(out, torch.Tensor) or out.device != dz.device or out.dtype != torch.float32:
        raise TypeError(f"out must be a float32 tensor on {dz.device}")
    if tuple(out.shape) != (n, m):
        raise ValueError(f"out must have shape {(n, m)}")
    _, _, ldg = _rows(out, "out")
    p, nb, keep = _scratch(ws, _size("dion3_linear_grad_weight_workspace_size", _ptr(dz), lddz, xp,
                                     ldx, sp, T, n, m), dz.device)
    _call("dion3_linear_grad_weight", dz.device, _ptr(dz), lddz, xp, ldx, sp, out.data_ptr(), ldg,
          int(bool(accumulate)), T, n, m, _DTYPES[dz.dtype], p, nb)
    return out


# ------------------------------------------------- the differentiable forms

def _as_rows(t):
    """A gradient as its producer left it, or contiguous where that has no
    rows that the library reads (an expanded gradient, a transposed one, a
    slice of very long rows): its layout is autograd's choice, not the user's."""
    try:
        if _rows(t, "gradient")[2] <= _MAX_LD:
            return t
    except ValueError:
        pass
    return t.contiguous()


class _RmsNormResidual(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, pack):
        y, h, rstd, p = add_rms_norm(x, weight, residual, eps, pack)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, rstd, weight)
        ctx.has_residual = residual is not None
        if residual is None:
            h = x.view_as(x)
        if p is None:
            return y, h, None, None
        ctx.mark_non_differentiable(p.q, p.scale)
        return y, h, p.q, p.scale

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh, _q, _s):
        h, rstd, weight = ctx.saved_tensors
        dx, dw = dh, None
        if dy is not None:
            need_x = ctx.needs_input_grad[0] or ctx.needs_input_grad[2]
            dx, dw = add_rms_norm_grad(_as_rows(dy), h, rstd, weight.contiguous(),
                                       None if dh is None else _as_rows(dh), need_dx=need_x,
                                       need_dw=ctx.needs_input_grad[1])
            if dw is not None:
                dw = dw.to(weight.dtype)
        return dx, dw, dx if ctx.has_residual else None, None, None


def rms_norm_residual(x, weight, residual=None, eps: float = 1e-6, pack: bool = False):
    """(y, h, packed) of ``add_rms_norm``, differentiable in x, weight and
    residual through y and h.  Kept for the backward pass: h and one fp32
    value per row.  ``packed`` (with ``pack``) is y in 8 bits, to be given to
    the layers that read y as their ``checkpoint``."""
    y, h, q, s = _RmsNormResidual.apply(x, weight, residual, eps, pack)
    return y, h, PackedF8(q, s, x.shape[-1], x.shape) if pack else None


def _accumulates(node):
    """What the running backward pass wants of the leaf behind ``node``, its
    AccumulateGrad: True to accumulate its gradient, False nothing (a pass
    restricted to other inputs), None its gradient as a value
    (``torch.autograd.grad`` with respect to the leaf).  What a custom function
    is told at its forward pass (``needs_input_grad``) knows no pass."""
    try:
        return torch._C._will_engine_execute_node(node)
    except RuntimeError:         # raised for a leaf whose gradient is the pass's result
        return None


class _LinearLayer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, act, checkpoint, into):
        w16 = w if w.dtype == x.dtype else w.to(x.dtype)
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        inner = need_x or need_w or need_b
        y, z = linear(x, w16, bias, act, residual, return_preact=inner and act != "none")
        full = checkpoint == "full" if isinstance(checkpoint, str) else False
        ctx.x = ctx.z = None                     # shapes of what is kept in 8 bits
        saved = [None] * 5                       # x or its q, its scale, z or its q, its scale, w
        if need_w:
            if full:
                saved[0] = x
            else:
                p = checkpoint if isinstance(checkpoint, PackedF8) else pack_f8(x)
                saved[0], saved[1], ctx.x = p.q, p.scale, (p.cols, p.shape)
        if z is not None:
            if full:
                saved[2] = z
            else:
                p = pack_f8(z)
                saved[2], saved[3], ctx.z = p.q, p.scale, (p.cols, p.shape)
        if need_x:
            saved[4] = w16
        ctx.save_for_backward(*saved)
        ctx.act, ctx.into, ctx.w = act, into, w if into is not None else None
        ctx.wtype, ctx.btype = w.dtype, bias.dtype if bias is not None else None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, xs, z, zs, w16 = ctx.saved_tensors
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        into = None
        if need_w and ctx.into is not None:
            wanted = _accumulates(ctx.next_functions[1][0])      # (x and w are inputs 0 and 1)
            need_w = wanted is not False
            into = ctx.into if wanted else None
        dx = dw = db = None
        if need_x or need_w or need_b:
            dyr = _as_rows(dy)
            if ctx.z is not None:
                z = PackedF8(z, zs, *ctx.z)
            dz, db = act_grad(dyr, z, ctx.act, bias=need_b)
            if need_x:
                dx = linear_grad_input(dz, w16)
            if need_w:
                xin = PackedF8(x, xs, *ctx.x) if ctx.x is not None else x
                if into is not None:
                    # (accumulate_grad, but a product that is refused names nothing)
                    m, captured = into._use(ctx.w)
                    linear_grad_weight(dz, xin, out=m, accumulate=True)
                    into._name(ctx.w, captured)
                else:
                    dw = linear_grad_weight(dz, xin).to(ctx.wtype)
            if db is not None:
                db = db.to(ctx.btype)
        return dx, dw, db, dy if need_r else None, None, None, None


def linear_layer(x, w, bias=None, act: str = "none", residual=None, checkpoint="f8", into=None):
    """y = act(x w^T + bias) + residual, differentiable in x, w, bias and
    residual.  ``w`` is of x's type or fp32 (then rounded to x's type for the
    products; its gradient is fp32).

    ``checkpoint``: what the backward pass reads of x and of the
    preactivation: "f8" (default) keeps both in 8 bits, a PackedF8 is x in 8
    bits as another layer or norm already keeps it (the preactivation is
    packed too), "full" keeps both as they are.  The forward result and the
    gradient of x are the same bits with every choice when act is "none".
    In 8 bits a value is off by up to 2^-4 of itself, and one below 4.4e-6 of
    the largest of its 32 columns may be 0: with "relu" such a preactivation
    passes no gradient.

    ``into``: a ``Dion3`` that steps w.  The weight gradient is then summed
    straight into w's momentum there, in the product's own epilogue; w gets no
    ``.grad``, and the next ``step()`` steps it.  What has been summed cannot
    be taken back by ``zero_grad()``.  This happens in the passes in which w's
    ``.grad`` would grow, and in no other: ``backward(inputs=[x])`` and
    ``torch.autograd.grad(y, x)`` leave the momentum alone, and
    ``torch.autograd.grad(y, w)`` returns the gradient.  What works on
    ``.grad`` does not see the sum: hooks of w get None and its post-accumulate
    hooks no ``.grad``; gradient clipping and reduction across processes pass
    it by; a scaled loss (fp16) enters the momentum scaled, cannot be unscaled
    there, and one overflow leaves infinities or NaN in it.  Train without
    ``into`` where you need any of these.

    Capturing into a graph: w's momentum must exist before (RuntimeError
    otherwise; an earlier step or ``into.momentum(w)`` makes it), and the
    optimizer does not see replays: call ``into.accumulate_grad(w)`` before
    each, on its stream, for the sum to be ordered behind earlier uses and for
    the next ``step()`` to step w.  torch's own
    rule for a captured backward pass holds here too: let no graph of the same
    leaves recorded outside the capture live (an earlier loss or output kept
    in a variable), since its end would have to join streams that the capture
    does not know."""
    if isinstance(checkpoint, PackedF8):
        if tuple(checkpoint.shape) != tuple(x.shape) or checkpoint.device != x.device:
            raise ValueError(f"checkpoint must stand for a tensor of shape {tuple(x.shape)} on "
                             f"{x.device}")
    elif checkpoint not in ("f8", "full"):
        raise ValueError('checkpoint must be "f8", "full" or a PackedF8')
    if not isinstance(w, torch.Tensor) or (w.dtype != x.dtype and w.dtype != torch.float32):
        raise TypeError(f"w must be {x.dtype} or float32")
    if into is not None:
        into.check_parameter(w)
    return _LinearLayer.apply(x, w, bias, residual, act, checkpoint, into)
