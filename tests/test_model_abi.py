"""Host-side checks of the entry points around the layers (embedding, heads,
log probabilities, gradient norm): arguments, sizes and workspaces.  No kernel
is launched: every call fails its checks first, or is over nothing.  CPU only."""
import ctypes

import pytest
import torch

import orthogonalizing_optimizer_amd as d3
from orthogonalizing_optimizer_amd import _lib, clip, model

OK, ERR_ARG, ERR_WS, ERR_UNSUP = 0, -1, -2, -3
P = 1 << 20              # a non-null, 256-aligned address that is never dereferenced
F32, BF16, F16 = 0, 1, 2
T, N, M = 40, 24, 16
BIG, LD, TOK = (1 << 20) + 1, (1 << 38) + 8, (1 << 24) + 1
NAN, INF = float("nan"), float("inf")


def call(fn, args, **change):
    a = dict(args)
    for k, v in change.items():
        assert k in a, k
        a[k] = v
    return getattr(d3.lib(), fn)(*a.values())


EMBED = dict(tok=P, bits=64, W=P, ldw=M, wtype=F32, Y=P, ldy=M, T=T, n=N, m=M, scale=1.0, dtype=BF16,
             stream=None)
EMBED_GRAD = dict(tok=P, bits=64, dY=P, lddy=M, dW=P, ldw=M, acc=0, T=T, n=N, m=M, scale=1.0,
                  dtype=BF16, ws=P, nb=1 << 30, stream=None)
LOGP = dict(X=P, ldx=N, tgt=P, bits=64, logp=P, stats=P, entropy=P, tl=P, ti=P, T=T, n=N, top=3,
            scale=1.0, dtype=BF16, ws=P, nb=1 << 30, stream=None)
LOGP_GRAD = dict(g=P, X=P, ldx=N, tgt=P, bits=64, stats=P, entropy=P, gh=P, dX=P, lddx=N, T=T, n=N,
                 scale=1.0, dtype=BF16, stream=None)
ALL = {"dion3_embedding": EMBED, "dion3_embedding_grad": EMBED_GRAD, "dion3_log_probs": LOGP,
       "dion3_log_probs_grad": LOGP_GRAD}


@pytest.mark.parametrize("fn", sorted(ALL))
def test_sizes_types_strides_and_pointers(fn):
    a = ALL[fn]
    assert call(fn, a, T=-1) == ERR_ARG and call(fn, a, T=TOK) == ERR_UNSUP
    wide = {k: LD - 8 for k in a if k.startswith("ld")}
    for k in ("n", "m"):
        if k in a:
            assert call(fn, a, **{k: 0}) == ERR_ARG
            assert call(fn, a, **wide, **{k: BIG}) == ERR_UNSUP
    for k in wide:
        assert call(fn, a, **{k: a[k] - 1}) == ERR_ARG and call(fn, a, **{k: LD}) == ERR_UNSUP
    for t in (-1, 3):
        assert call(fn, a, dtype=t) == ERR_ARG
    for b in (0, 16, 63):
        assert call(fn, a, bits=b) == ERR_ARG
    for s in (NAN, INF, -INF):
        assert call(fn, a, scale=s) == ERR_ARG
    for k, v in a.items():                      # odd addresses
        if v == P and k != "ws":
            assert call(fn, a, **{k: P + 1}) == ERR_ARG, k
    assert call(fn, a, T=0) == OK if fn != "dion3_embedding_grad" else call(fn, a, T=0, acc=1) == OK


NEEDED = {"dion3_embedding": "tok W Y", "dion3_embedding_grad": "tok dY dW",
          "dion3_log_probs": "X stats tl ti logp tgt", "dion3_log_probs_grad": "X stats dX g tgt entropy"}


@pytest.mark.parametrize("fn", sorted(ALL))
def test_missing_pointers(fn):
    for k in NEEDED[fn].split():
        assert call(fn, ALL[fn], **{k: None}) == ERR_ARG, k


def test_combinations():
    assert call("dion3_embedding", EMBED, wtype=F16) == ERR_ARG
    assert call("dion3_embedding", EMBED, wtype=BF16, dtype=F32) == ERR_ARG
    for s in (0.0, -1.0):
        assert call("dion3_log_probs", LOGP, scale=s) == ERR_ARG
        assert call("dion3_log_probs_grad", LOGP_GRAD, scale=s) == ERR_ARG
    assert call("dion3_log_probs", LOGP, top=-1) == ERR_ARG
    assert call("dion3_log_probs", LOGP, top=N + 1) == ERR_ARG
    assert call("dion3_log_probs", LOGP, top=65, n=100, ldx=100) == ERR_UNSUP
    assert call("dion3_log_probs_grad", LOGP_GRAD, g=None, tgt=None, gh=None) == ERR_ARG


def size(fn, *args):
    out = ctypes.c_size_t(12345)
    st = getattr(d3.lib(), fn)(*args, ctypes.byref(out))
    return st, out.value


def test_workspaces():
    for fn, a, args in (("dion3_embedding_grad", EMBED_GRAD, (T, N, M)),
                        ("dion3_log_probs", LOGP, (T, N, 3))):
        st, nb = size(fn + "_workspace_size", *args)
        assert st == OK and nb > 0
        for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
            assert call(fn, a, **change) == ERR_WS
        assert getattr(d3.lib(), fn + "_workspace_size")(*args, None) == ERR_ARG
        assert size(fn + "_workspace_size", 0, *args[1:]) == (OK, 0)
    # counted places, then places by digits
    small, large = (size("dion3_embedding_grad_workspace_size", t, N, M)[1] for t in (8192, 8193))
    assert large > small + 2 * 4 * 8193
    assert size("dion3_log_probs_workspace_size", T, N, 65)[0] == ERR_ARG
    assert size("dion3_log_probs_workspace_size", T, 100, 65)[0] == ERR_UNSUP


def heads(**change):
    a = dict(X=P, ldx=4 * M, hsx=M, w=P, dY=P, lddy=4 * M, hsdy=M, Y=P, ldy=4 * M, hsy=M, heads=4)
    a.update(change)
    return _lib.HeadsDesc(**a)


def rope(q, k=None, grad=False, ws=P, nb=1 << 30, **change):
    a = dict(freqs=P, pos=P, bits=64, T=T, D=M, r=8, il=0, eps=1e-6, wtype=F32, dtype=BF16, dw=P)
    a.update(change)
    q, k = ctypes.byref(q) if q else None, ctypes.byref(k) if k else None
    if not grad:
        return d3.lib().dion3_qk_norm_rope(q, k, a["freqs"], a["pos"], a["bits"], a["T"], a["D"], a["r"],
                                           a["il"], a["eps"], a["wtype"], a["dtype"], None)
    return d3.lib().dion3_qk_norm_rope_grad(q, k, a["freqs"], a["pos"], a["bits"], a["dw"], a["T"],
                                            a["D"], a["r"], a["il"], a["eps"], a["wtype"], a["dtype"],
                                            ws, nb, None)


@pytest.mark.parametrize("grad", [False, True])
def test_heads(grad):
    def r(q=heads(), k=heads(), **kw):
        return rope(q, k, grad, **kw)

    assert rope(None, heads(), grad) == ERR_ARG
    for bad in (dict(T=-1), dict(D=0), dict(r=7), dict(r=-2), dict(r=18), dict(il=2), dict(bits=16),
                dict(eps=-1.0), dict(eps=NAN), dict(wtype=F16), dict(dtype=F32), dict(freqs=None),
                dict(pos=None), dict(pos=P + 4), dict(freqs=P + 4), dict(r=M, D=M - 2)):
        assert r(**bad) == ERR_ARG, bad
    assert r(T=TOK) == ERR_UNSUP
    wide = heads(ldx=1 << 13, hsx=1 << 11, lddy=1 << 13, hsdy=1 << 11, ldy=1 << 13, hsy=1 << 11)
    assert r(q=wide, k=wide, D=1025) == ERR_UNSUP
    assert r(q=wide, k=wide, D=1023, r=1022) == ERR_UNSUP      # 65 pieces of 16 columns
    for bad in (dict(X=None), dict(w=None), dict(X=P + 1), dict(w=P + 2), dict(heads=0), dict(ldx=M - 1),
                dict(hsx=M - 1), dict(ldy=M - 1), dict(hsy=M - 1), dict(Y=P + 1)):
        assert r(q=heads(**bad)) == ERR_ARG, bad
        assert r(k=heads(**bad)) == ERR_ARG, bad
    for bad in (dict(heads=65537), dict(ldx=(1 << 38) + 1), dict(hsx=(1 << 38) + 1)):
        assert r(q=heads(**bad)) == ERR_UNSUP, bad
    if grad:
        assert r(q=heads(dY=None)) == ERR_ARG and r(q=heads(hsdy=M - 1)) == ERR_ARG
        assert r(q=heads(Y=None), k=heads(Y=None), dw=None) == ERR_ARG
        st, nb = size("dion3_qk_norm_rope_grad_workspace_size", T, 4, 4, M, 8, 0)
        assert st == OK and nb >= 2 * M * 4
        for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
            assert r(**change) == ERR_WS
        assert size("dion3_qk_norm_rope_grad_workspace_size", T, 0, 4, M, 8, 0)[0] == ERR_ARG
        assert r(T=0, dw=None) == OK
    else:
        assert r(q=heads(Y=None)) == ERR_ARG
        assert r(T=0) == OK


def grads(*descs):
    return (_lib.GradDesc * len(descs))(*[_lib.GradDesc(**dict(dict(G=P, M=None, rows=4, cols=8, ldg=8,
                                                                    ldm=8, dtype=F32), **d)) for d in descs])


def test_gradient_norm():
    lib = d3.lib()

    def norm(a, count=None, scale=1.0, norm=P, norms=None, ws=P, nb=1 << 30):
        return lib.dion3_grad_norm(a, len(a) if count is None else count, scale, norm, norms, ws, nb, None)

    def clipped(a, most=1.0, scale=1.0, norm=P, ws=P, nb=1 << 30):
        return lib.dion3_clip_grad_norm(a, len(a), most, scale, norm, ws, nb, None)

    for f in (norm, clipped):
        for bad in (dict(rows=-1), dict(cols=-1), dict(G=None), dict(G=P + 2), dict(dtype=3), dict(ldg=7)):
            assert f(grads({}, bad)) == ERR_ARG, bad
        for bad in (dict(rows=1 << 20, cols=1 << 20, ldg=1 << 20), dict(rows=1, cols=(1 << 38) + 1)):
            assert f(grads(bad)) == ERR_UNSUP
        for s in (0.0, -1.0, NAN, INF):
            assert f(grads({}), scale=s) == ERR_ARG
        nb = size("dion3_grad_norm_workspace_size", grads({}), 1)[1]
        for change in (dict(ws=None), dict(ws=P + 128), dict(nb=nb - 1)):
            assert f(grads({}), **change) == ERR_WS
        assert f(grads({}), norm=P + 2) == ERR_ARG
    assert norm(grads({}), norm=None) == ERR_ARG and norm(grads({}), norms=P + 1) == ERR_ARG
    assert norm(grads({}), count=-1) == ERR_ARG and norm(None, count=1) == ERR_ARG
    assert norm(grads({}), count=(1 << 20) + 1) == ERR_UNSUP
    for most in (-1.0, NAN):
        assert clipped(grads({}), most=most) == ERR_ARG
    assert clipped(grads(dict(M=P, ldm=7))) == ERR_ARG and clipped(grads(dict(M=P + 2))) == ERR_ARG
    # nothing to do, nothing launched
    assert clipped(grads(dict(G=None, rows=0)), norm=None) == OK
    assert size("dion3_grad_norm_workspace_size", grads(dict(G=None, cols=0)), 1) == (OK, 0)


def test_binding_refuses_host_tensors():
    x, t = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    v, h = torch.ones(8), torch.zeros(4, 2, 8, dtype=torch.bfloat16)
    for f in (lambda: d3.embedding(t, x), lambda: d3.embedding_grad(t, x, 4), lambda: d3.log_probs(x, t),
              lambda: d3.log_probs_grad(v, x, t, v), lambda: d3.grad_norm([x]),
              lambda: d3.clip_grad_norm([x], 1.0), lambda: d3.token_log_probs(x, t),
              lambda: d3.qk_norm_rope(h, h, v, v, t, v.double()), lambda: d3.embedding_layer(t, x)):
        with pytest.raises(TypeError):
            f()


def test_layouts_of_gradients():
    whole = clip._whole
    t = torch.zeros(4, 6)
    assert whole(t) and whole(t.t()) and whole(t[1:]) and whole(t[:, None].transpose(0, 2))
    assert not whole(t[:, 1:]) and not whole(t[:, ::2]) and not whole(t[:1].expand(4, 6))
    assert whole(torch.zeros(3, 1, 2).expand(3, 1, 2)) and whole(torch.zeros(()))


def test_layouts_of_heads():
    x = torch.zeros(2, 5, 4, 8)
    assert model._heads(x, "x") == (10, 32, 4, 8, 8)
    assert model._heads(x[:, :, 1:3], "x") == (10, 32, 2, 8, 8)
    assert model._heads(torch.zeros(4, 10, 8).transpose(0, 1), "x") == (10, 8, 4, 80, 8)
    assert model._heads(torch.zeros(0, 4, 8), "x")[0] == 0
    for bad in (x.transpose(2, 3), x.transpose(1, 2).transpose(0, 1), torch.zeros(3, 1, 8).expand(3, 4, 8),
                torch.zeros(8)):
        with pytest.raises(ValueError):
            model._heads(bad, "x")
