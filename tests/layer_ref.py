"""Plain 64-bit forms of the layer operators (on the CPU, from the formulas)
and the error bounds their tests use.

Bounds count roundings: U[t] is half a step of type t relative to the value,
EPS32 that of fp32.  A sum of N fp32 terms in any order is off by at most
N EPS32 times the sum of their magnitudes (first order; N stands for the
longest chain of additions a term goes through, at most the number of terms).
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
EPS32 = 2.0 ** -24
BLOCK = 32


def d(t):
    return t.detach().cpu().double()


def close(got, want, bound, what=""):
    """|got - want| <= bound elementwise."""
    err = (d(got) - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / bound.clamp_min(1e-300)).nan_to_num(1e9).max()):.3g} "
                           "times the bound")


def rounded(want, t, extra=0.0):
    """Bound of a value rounded once to type t, after an error `extra`."""
    return (want.abs() + extra) * U[t] + extra + TINY[t]


# ------------------------------------------------------------------- formulas

def act(z, name):
    if name == "relu":
        return z.clamp_min(0)
    if name == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if name == "gelu_tanh":
        return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.special.expit(z)
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return (torch.special.erfc(-z / math.sqrt(2)) / 2
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        s = torch.special.expit(u)
        return s + z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.special.expit(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# The functions' own error in fp32, relative to |z| (values) or to 1 (slopes):
# the argument of exp (at most 3 roundings of a value up to about 2 |z| +
# |z|^3 / 10, of which only the range where sigmoid is not 0 or 1 counts: an
# argument |u| <= 20 off by 4 EPS32 |u| moves sigmoid by at most 4 EPS32 |u|
# e^-|u| <= 2 EPS32), exp and the division (4 EPS32), and the two products.
ACT_EPS = 32 * EPS32


def e4m3_values():
    """The 256 values of the 8-bit type (index = byte)."""
    out = []
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            v = float("nan")
        elif e == 0:
            v = m * 2.0 ** -9
        else:
            v = (8 + m) * 2.0 ** (e - 10)
        out.append(-v if s else v)
    return torch.tensor(out, dtype=torch.float64)


def pack(x):
    """(bytes [T, mp] uint8, scale [T, mp / 32] uint8) of x (CPU, any type):
    the nearest representable value by search, ties to the even byte."""
    t = x.dtype
    v = d(x)
    T, m = v.shape
    mp = -(-m // BLOCK) * BLOCK
    v = torch.cat([v, torch.zeros(T, mp - m, dtype=torch.float64)], 1).view(T, -1, BLOCK)
    amax = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(2)
    mant, ex = torch.frexp(amax)
    e = torch.where(amax == 0, torch.full_like(ex, -127), ex - 9 + (mant > 0.875)).clamp_min(-127)
    last = 8 if t == torch.float16 else 120
    lim = torch.where(e == last, 240.0, 448.0).double().unsqueeze(2)
    u = torch.ldexp(v, -e.unsqueeze(2).double())
    fin = torch.isfinite(u)
    a = torch.minimum(torch.where(fin, u.abs(), torch.zeros_like(u)), lim)
    grid = e4m3_values()[:127]                      # 0 .. 448, ascending
    hi = torch.searchsorted(grid, a.contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    dl, dh = a - grid[lo], grid[hi] - a
    b = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    b = torch.where(torch.signbit(u), b + 128, b)
    b = torch.where(fin, b, torch.full_like(b, 127))
    return b.view(T, mp).to(torch.uint8), (e + 127).to(torch.uint8)


def unpack(q, s):
    """float64 values of (bytes, scale)."""
    v = e4m3_values()[q.long()].view(q.shape[0], -1, BLOCK)
    return torch.ldexp(v, s.double().unsqueeze(2) - 127).view(q.shape)
