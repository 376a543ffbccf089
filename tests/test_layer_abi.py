"""Host-side checks of the layer operators' entry points: argument, size and
workspace validation.  No kernel is launched: every call here fails its checks
before the first launch, or is over no tokens.  CPU only."""
import ctypes

import pytest
import torch

import orthogonalizing_optimizer_amd as d3

OK, ERR_ARG, ERR_WS, ERR_UNSUP = 0, -1, -2, -3
P = 1 << 20              # a non-null, 256-aligned address that is never dereferenced
F32, BF16, F16 = 0, 1, 2
T, N, M = 40, 24, 16
BIG = (1 << 20) + 1      # past DION3_MAX_DIM
LD = (1 << 21) + 8       # past the largest row stride
TOK = (1 << 24) + 1      # past DION3_MAX_TOKENS


def call(fn, args, **change):
    a = dict(args)
    for k, v in change.items():
        assert k in a, k
        a[k] = v
    return getattr(d3.lib(), fn)(*a.values())


NORM = dict(X=P, ldx=M, R=P, ldr=M, w=P, wtype=F32, H=P, ldh=M, Y=P, ldy=M, Q=P, S=P, rstd=P, T=T,
            m=M, eps=1e-6, dtype=BF16, stream=None)
NORM_GRAD = dict(dY=P, lddy=M, H=P, ldh=M, rstd=P, w=P, wtype=F32, dH=P, lddh=M, dX=P, lddx=M, dw=P,
                 T=T, m=M, dtype=BF16, ws=P, nb=1 << 30, stream=None)
PACK = dict(X=P, ldx=M, Q=P, S=P, T=T, m=M, dtype=BF16, stream=None)
UNPACK = dict(Q=P, S=P, Y=P, ldy=M, T=T, m=M, dtype=BF16, stream=None)
LINEAR = dict(X=P, ldx=M, W=P, ldw=M, bias=P, btype=F32, R=P, ldr=N, Y=P, ldy=N, Z=P, ldz=N, T=T, n=N,
              m=M, act=1, dtype=BF16, ws=P, nb=1 << 30, stream=None)
ACT_GRAD = dict(dY=P, lddy=N, Z=P, ldz=N, ZQ=None, ZS=None, dZ=P, lddz=N, db=P, T=T, n=N, act=1,
                dtype=BF16, ws=P, nb=1 << 30, stream=None)
GRAD_INPUT = dict(dZ=P, lddz=N, W=P, ldw=M, R=P, ldr=M, dX=P, lddx=M, T=T, n=N, m=M, dtype=BF16, ws=P,
                  nb=1 << 30, stream=None)
GRAD_WEIGHT = dict(dZ=P, lddz=N, X=P, ldx=M, S=None, G=P, ldg=M, acc=0, T=T, n=N, m=M, dtype=BF16,
                   ws=P, nb=1 << 30, stream=None)
ALL = {"dion3_add_rms_norm": NORM, "dion3_add_rms_norm_grad": NORM_GRAD, "dion3_pack_f8": PACK,
       "dion3_unpack_f8": UNPACK, "dion3_linear": LINEAR, "dion3_act_grad": ACT_GRAD,
       "dion3_linear_grad_input": GRAD_INPUT, "dion3_linear_grad_weight": GRAD_WEIGHT}


@pytest.mark.parametrize("fn", sorted(ALL))
def test_sizes_types_strides_and_pointers(fn):
    a = ALL[fn]
    sides = [k for k in ("n", "m") if k in a]
    assert call(fn, a, T=-1) == ERR_ARG
    assert call(fn, a, T=TOK) == ERR_UNSUP
    for k in sides:
        assert call(fn, a, **{k: 0}) == ERR_ARG
        big = {"n": BIG, "m": BIG}
        assert call(fn, a, **{k: big[k]}) in (ERR_ARG, ERR_UNSUP)
    wide = {k: LD for k in a if k.startswith("ld")}
    assert call(fn, a, **{k: BIG for k in sides}, **wide) == ERR_UNSUP
    for k in wide:
        assert call(fn, a, **{k: LD}) == ERR_UNSUP, k
        assert call(fn, a, **{k: 0}) == ERR_ARG, k
        assert call(fn, a, **{k: a[k] - 1}) == ERR_ARG, k
    for t in (-1, 3, 7):
        assert call(fn, a, dtype=t) == ERR_ARG
    for k, v in a.items():                      # odd addresses
        if v == P and k not in ("S", "ws"):
            assert call(fn, a, **{k: P + 1}) == ERR_ARG, k
    # more than 2^31 workgroups of 256 chunks
    assert call(fn, a, T=1 << 24, **{k: 1 << 20 for k in sides},
                **{k: 1 << 20 for k in wide}) == ERR_UNSUP


NEEDED = {"dion3_add_rms_norm": "X w", "dion3_add_rms_norm_grad": "dY H rstd w",
          "dion3_pack_f8": "X Q S", "dion3_unpack_f8": "Q S Y", "dion3_linear": "X W Y",
          "dion3_act_grad": "dY", "dion3_linear_grad_input": "dZ W dX",
          "dion3_linear_grad_weight": "dZ X G"}


@pytest.mark.parametrize("fn", sorted(ALL))
def test_missing_pointers(fn):
    for k in NEEDED[fn].split():
        assert call(fn, ALL[fn], **{k: None}) == ERR_ARG, k


@pytest.mark.parametrize("fn", sorted(ALL))
def test_no_tokens_need_no_device(fn):
    """T = 0: nothing to do, so nothing is checked against a device either
    (the gradients' zeros apart)."""
    a = ALL[fn]
    if fn in ("dion3_add_rms_norm_grad", "dion3_act_grad"):
        name = "dw" if "dw" in a else "db"
        assert call(fn, a, T=0, **{name: None}) == OK
    elif fn == "dion3_linear_grad_weight":
        assert call(fn, a, T=0, acc=1) == OK
    else:
        assert call(fn, a, T=0) == OK


def test_norm_combinations():
    f = "dion3_add_rms_norm"
    assert call(f, NORM, R=None) == ERR_ARG and call(f, NORM, H=None) == ERR_ARG
    assert call(f, NORM, Q=None) == ERR_ARG and call(f, NORM, S=None) == ERR_ARG
    assert call(f, NORM, Y=None, Q=None, S=None) == ERR_ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(f, NORM, eps=eps) == ERR_ARG
    assert call(f, NORM, wtype=F16) == ERR_ARG and call(f, NORM, dtype=F32) == ERR_ARG
    g = "dion3_add_rms_norm_grad"
    assert call(g, NORM_GRAD, dX=None, dw=None) == ERR_ARG
    assert call(g, NORM_GRAD, wtype=F16) == ERR_ARG and call(g, NORM_GRAD, dtype=F32) == ERR_ARG


def test_product_combinations():
    assert call("dion3_linear", LINEAR, act=5) == ERR_ARG
    assert call("dion3_linear", LINEAR, act=-1) == ERR_ARG
    assert call("dion3_linear", LINEAR, btype=F16) == ERR_ARG
    assert call("dion3_linear", LINEAR, dtype=F32) == ERR_ARG
    assert call("dion3_act_grad", ACT_GRAD, act=9) == ERR_ARG
    assert call("dion3_act_grad", ACT_GRAD, Z=None) == ERR_ARG           # no z at all
    assert call("dion3_act_grad", ACT_GRAD, ZQ=P, ZS=P) == ERR_ARG       # both forms
    assert call("dion3_act_grad", ACT_GRAD, Z=None, ZQ=P) == ERR_ARG     # half a form
    assert call("dion3_act_grad", ACT_GRAD, dZ=None, db=None) == ERR_ARG
    assert call("dion3_linear_grad_weight", GRAD_WEIGHT, S=P, X=P + 4) == ERR_ARG
    assert call("dion3_linear_grad_weight", GRAD_WEIGHT, dtype=F32) == ERR_ARG


def size(fn, *args):
    out = ctypes.c_size_t(12345)
    st = getattr(d3.lib(), fn)(*args, ctypes.byref(out))
    return st, out.value


def test_workspaces():
    st, nb = size("dion3_add_rms_norm_grad_workspace_size", T, M)
    assert st == OK and nb >= M * 4
    for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
        assert call("dion3_add_rms_norm_grad", NORM_GRAD, **change) == ERR_WS
    st, nb = size("dion3_act_grad_workspace_size", T, N)
    assert st == OK and nb >= N * 4
    for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
        assert call("dion3_act_grad", ACT_GRAD, **change) == ERR_WS
    # an operand off its alignment is read as it is, but rows of fewer than 8
    # elements are copied: the workspace holds them
    odd = P + 2
    for fn in ("dion3_linear_workspace_size", "dion3_linear_grad_input_workspace_size"):
        assert size(fn, odd, 24, P, 24, T, 24, 24) == size(fn, P, 24, P, 24, T, 24, 24) == (OK, 0)
    st, nb = size("dion3_linear_workspace_size", odd, 7, P, 8, T, N, 7)
    assert st == OK and nb >= (T + N) * 8 * 2
    for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
        assert call("dion3_linear", LINEAR, X=odd, ldx=7, ldw=8, m=7, **change) == ERR_WS
    st, nb = size("dion3_linear_grad_input_workspace_size", odd, 7, P, M, T, 7, M)
    assert st == OK and nb >= T * 8 * 2
    assert call("dion3_linear_grad_input", GRAD_INPUT, dZ=odd, lddz=7, n=7, nb=nb - 1) == ERR_WS
    # few tiles and many tokens: split, fp32 parts in the workspace
    st, nb = size("dion3_linear_grad_weight_workspace_size", P, 128, P, 512, None, 16384, 128, 512)
    assert st == OK and nb >= 2 * 128 * 512 * 4
    st, nb8 = size("dion3_linear_grad_weight_workspace_size", P, 128, P, 0, P, 16384, 128, 512)
    assert st == OK and nb8 == nb
    big = dict(GRAD_WEIGHT, lddz=128, ldx=512, ldg=512, T=16384, n=128, m=512)
    for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
        assert call("dion3_linear_grad_weight", big, **change) == ERR_WS
    for fn, a in (("dion3_add_rms_norm_grad_workspace_size", (T, 0)),
                  ("dion3_act_grad_workspace_size", (-1, N)),
                  ("dion3_linear_workspace_size", (P, M - 1, P, M, T, N, M))):
        assert size(fn, *a) == (ERR_ARG, 12345)
        assert getattr(d3.lib(), fn)(*a, None) == ERR_ARG


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(8, 8, dtype=torch.bfloat16)
    v = torch.ones(8)
    for f in (lambda: d3.linear(x, w), lambda: d3.linear_grad_input(x, w),
              lambda: d3.linear_grad_weight(x, x), lambda: d3.act_grad(x, x, "relu"),
              lambda: d3.pack_f8(x), lambda: d3.add_rms_norm(x, v),
              lambda: d3.add_rms_norm_grad(x, x, v[:4], v), lambda: d3.unpack_f8(x),
              lambda: d3.PackedF8(x.to(torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8), 8)):
        with pytest.raises(TypeError):
            f()


def test_most_elements():
    """A matrix of up to 2^38 elements passes the checks, a larger one does not."""
    t, m = 1 << 24, 1 << 14
    for fn in ("dion3_add_rms_norm_grad_workspace_size", "dion3_act_grad_workspace_size"):
        assert size(fn, t, m)[0] == OK
        assert size(fn, t, m + 1) == (ERR_UNSUP, 12345)
    for fn in ("dion3_linear_workspace_size", "dion3_linear_grad_input_workspace_size"):
        assert size(fn, P, m, P, m, t, 64 if "input" not in fn else m, m)[0] == OK
        for T_, n_, m_ in ((t, m + 1, 64), (t, 64, m + 1), (1, 1 << 20, (1 << 18) + 1)):
            assert size(fn, P, 1 << 20, P, 1 << 20, T_, n_, m_) == (ERR_UNSUP, 12345)
