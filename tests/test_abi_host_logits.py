"""Host-side refusals of the norm with the residual's addition, the token log
probabilities and the distillation (no GPU: every call below returns from host
validation), and the binding's own checks."""
import ctypes as C

import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from elementwise_epilogues_transformer_gb300 import build as B

OK, NULL, SHAPE, DTYPE, PROB, ALIAS, CUDA, DEVICE, WORKSPACE, VALUE = range(10)
INF, NAN = float("inf"), float("nan")

# Fake, never-dereferenced device addresses, far apart.
X, R, W, Y, H, S, Q, D = (0x100000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def L():
    B.build()
    return mfx.lib()


def fwd(L, **k):
    a = {**dict(xdt=1, rdt=0, wdt=1, rows=4, cols=64, x=X, r=R, w=W, eps=1e-6, off=0.0, y=Y, h=H, s=S), **k}
    return L.mfx_add_rmsnorm_fwd(a["xdt"], a["rdt"], a["wdt"], a["rows"], a["cols"], a["x"], a["r"], a["w"], a["eps"],
                                 a["off"], a["y"], a["h"], a["s"], None)


def quant(L, **k):
    a = {**dict(xdt=1, rdt=0, wdt=1, rows=4, cols=64, x=X, r=R, w=W, eps=1e-6, off=0.0, qdt=2, group=32, sdt=0, q=Q, sc=D,
                h=H, s=S), **k}
    return L.mfx_add_rmsnorm_quant_fwd(a["xdt"], a["rdt"], a["wdt"], a["rows"], a["cols"], a["x"], a["r"], a["w"], a["eps"],
                                       a["off"], a["qdt"], a["group"], a["sdt"], a["q"], a["sc"], a["h"], a["s"], None)


def bwd(L, **k):
    a = {**dict(xdt=1, rdt=0, wdt=1, rows=4, cols=64, dy=X, h=H, s=S, w=W, off=0.0, dh=R, dx=Y, dr=D, dw=Q,
                ws=0x1000000000, size=1 << 24), **k}
    n = C.c_size_t(a["size"]) if a["size"] is not None else None
    st = L.mfx_add_rmsnorm_bwd(a["xdt"], a["rdt"], a["wdt"], a["rows"], a["cols"], a["dy"], a["h"], a["s"], a["w"], a["off"],
                               a["dh"], a["dx"], a["dr"], a["dw"], a["ws"], C.byref(n) if n is not None else None, None)
    return st, n.value if n is not None else None


def test_norm_validation(L):
    for call in (fwd, quant, lambda L, **k: bwd(L, **{("dy" if n == "x" else n): v for n, v in k.items()})[0]):
        for k in ("xdt", "rdt", "wdt"):
            assert call(L, **{k: 2}) == DTYPE and call(L, **{k: -1}) == DTYPE
        for k, v in (("rows", -1), ("cols", -1), ("rows", 2 ** 60), ("cols", 2 ** 31)):
            assert call(L, **{k: v}) == SHAPE, (k, v)
        for v in (INF, -INF, NAN):
            assert call(L, off=v) == VALUE
        assert call(L, x=None) == NULL
    for call in (fwd, quant):
        for v in (-1e-6, NAN, INF):
            assert call(L, eps=v) == VALUE
        assert call(L, r=None) == NULL                       # h without a residual
        assert call(L, rows=0, x=None, r=None, w=None) == OK and call(L, cols=0, x=None) == OK
        assert call(L, s=W) == ALIAS and call(L, h=R + 4) == ALIAS and call(L, w=H + 8) == ALIAS
        assert call(L, s=X + 16) == ALIAS and call(L, h=X) == ALIAS  # other sizes than x's
    assert fwd(L, y=None) == NULL and fwd(L, y=X + 2) == ALIAS and fwd(L, y=H) == ALIAS and fwd(L, y=R) == ALIAS
    n = 4 * 64
    assert quant(L, q=None) == NULL and quant(L, sc=None) == NULL
    assert quant(L, q=X) == ALIAS and quant(L, sc=X) == ALIAS and quant(L, sc=Q + n - 1) == ALIAS and quant(L, sc=R) == ALIAS
    for v in (1, 16, 64, 256, -32):
        assert quant(L, group=v) == VALUE
    for k in ("qdt", "sdt"):
        for v in (1, 5, -1):
            assert quant(L, **{k: v}) == DTYPE
    assert quant(L, qdt=0) == DTYPE and quant(L, qdt=4) == DTYPE and quant(L, sdt=2) == DTYPE


def test_norm_bwd_validation(L):
    for k in ("dy", "h", "s"):
        assert bwd(L, **{k: None})[0] == NULL
    assert bwd(L, dx=None, dr=None)[0] == NULL and bwd(L, w=None)[0] == NULL  # dweight without a weight
    assert bwd(L, dx=X + 2)[0] == ALIAS and bwd(L, dr=X)[0] == ALIAS and bwd(L, dx=H)[0] == ALIAS
    assert bwd(L, dx=D)[0] == ALIAS and bwd(L, dw=W)[0] == ALIAS and bwd(L, dw=X)[0] == ALIAS and bwd(L, dr=S)[0] == ALIAS
    assert bwd(L, ws=X)[0] == ALIAS and bwd(L, ws=Y + 16)[0] == ALIAS
    st, need = bwd(L, ws=None, size=0)
    assert st == OK and need > 0 and need % (64 * 4) == 0
    assert bwd(L, ws=None, size=0, dy=None, h=None, s=None, dx=None, dr=None) == (OK, need)
    assert bwd(L, size=need - 1)[0] == WORKSPACE and bwd(L, ws=0x1000000008)[0] == WORKSPACE
    assert bwd(L, ws=None, size=None)[0] == NULL
    assert bwd(L, ws=None, size=0, dw=None) == (OK, 0)       # nothing to sum
    st, longer = bwd(L, ws=None, size=0, dw=None, cols=40000)
    assert st == OK and longer == 4 * 4                      # the rows' own sums
    assert bwd(L, ws=None, size=None, dw=None, cols=40000)[0] == NULL
    assert bwd(L, ws=None, size=9, rows=0) == (OK, 0)


def lp(L, **k):
    a = {**dict(dt=1, rows=4, v=100, ld=100, z=X, bits=64, t=R, scale=1.0, top=3, lp=Y, e=H, tv=S, ti=Q, st=D, ws=None,
                size=None), **k}
    n = C.c_size_t(a["size"]) if a["size"] is not None else None
    st = L.mfx_token_logprobs_fwd(a["dt"], a["rows"], a["v"], a["ld"], a["z"], a["bits"], a["t"], a["scale"], a["top"],
                                  a["lp"], a["e"], a["tv"], a["ti"], a["st"], a["ws"], C.byref(n) if n is not None else None,
                                  None)
    return (st, n.value) if n is not None else st


def lpb(L, **k):
    a = {**dict(dt=1, rows=4, v=100, ld=100, g=Y, ge=H, z=X, bits=64, t=R, st=S, scale=1.0, d=D, ldo=100), **k}
    return L.mfx_token_logprobs_bwd(a["dt"], a["rows"], a["v"], a["ld"], a["g"], a["ge"], a["z"], a["bits"], a["t"], a["st"],
                                    a["scale"], a["d"], a["ldo"], None)


def test_logprobs_validation(L):
    for call in (lp, lpb):
        assert call(L, dt=2) == DTYPE and call(L, bits=16) == DTYPE and call(L, bits=0) == DTYPE
        for k, v in (("rows", -1), ("v", -1), ("ld", 99), ("rows", 2 ** 60), ("v", 2 ** 31)):
            assert call(L, **{k: v}) == SHAPE, (k, v)
        for v in (0.0, -1.0, NAN, INF, 3e38):
            assert call(L, scale=v) == VALUE
        assert call(L, z=None) == NULL and call(L, t=None) == NULL
        assert call(L, rows=0, z=None, t=None) == OK
    for v in (-1, 65):
        assert lp(L, top=v) == VALUE
    for k in ("lp", "e", "tv", "ti"):
        assert lp(L, **{k: None}) == NULL
    assert lp(L, lp=H) == ALIAS and lp(L, tv=Q) == ALIAS and lp(L, st=X + 8) == ALIAS and lp(L, lp=R) == ALIAS
    assert lp(L, ti=X + (3 * 100 + 99) * 2) == ALIAS          # the last logit
    # few rows need no workspace, many do for alternatives
    assert lp(L, size=7, rows=1) == (OK, 0) and lp(L, size=7, top=0, rows=10 ** 5) == (OK, 0) and lp(L, size=7, rows=0) == (OK, 0)
    st, need = lp(L, size=0, rows=10 ** 5, lp=None, e=None, z=None, t=None)
    assert st == OK and need >= 10 ** 5 * 4 * 34
    many = dict(rows=10 ** 5, z=X, t=R << 4, lp=Y << 4, e=H << 4, tv=S << 4, ti=Q << 4, st=D << 4)
    assert lp(L, **many) == NULL
    assert lp(L, **many, ws=W << 12, size=need - 1)[0] == WORKSPACE
    assert lp(L, **many, ws=(W << 12) + 8, size=need)[0] == WORKSPACE
    assert lp(L, **many, ws=Y << 4, size=need)[0] == ALIAS


def test_logprobs_bwd_validation(L):
    assert lpb(L, g=None, ge=None) == NULL and lpb(L, st=None) == NULL and lpb(L, d=None) == NULL
    assert lpb(L, ldo=99) == SHAPE
    assert lpb(L, v=0, ld=0, ldo=0, z=None, t=None, d=None) == OK
    assert lpb(L, d=X + 2) == ALIAS and lpb(L, d=S) == ALIAS and lpb(L, d=R) == ALIAS and lpb(L, d=Y) == ALIAS and lpb(L, d=H) == ALIAS
    assert lpb(L, d=X, ldo=104) == ALIAS                      # the same buffer, other rows


def args(a):
    return a["dt"], a["tdt"], a["rows"], a["v"], a["ld"], a["k"]


BASE = dict(dt=1, tdt=0, rows=4, v=100, ld=100, k=8, z=X, bits=64, i=R, t=W, lse=None, g=H, st=S, loss=Y, scale=1.0, d=D,
            ldo=100)


def dfwd(L, **k):
    a = {**BASE, **k}
    return L.mfx_topk_distill_fwd(*args(a), a["z"], a["bits"], a["i"], a["t"], a["lse"], a["scale"], a["loss"], a["st"], None)


def dbwd(L, **k):
    a = {**BASE, **k}
    return L.mfx_topk_distill_bwd(*args(a), a["g"], a["z"], a["bits"], a["i"], a["t"], a["st"], a["scale"], a["d"], a["ldo"],
                                  None)


def dboth(L, **k):
    a = {**BASE, **k}
    return L.mfx_topk_distill_fwd_bwd(*args(a), a["z"], a["bits"], a["i"], a["t"], a["lse"], a["g"], a["scale"], a["loss"],
                                      a["d"], a["ldo"], None)


def test_distill_validation(L):
    for call in (dfwd, dbwd, dboth):
        assert call(L, dt=3) == DTYPE and call(L, tdt=2) == DTYPE and call(L, bits=8) == DTYPE
        for k, v in (("rows", -1), ("v", -1), ("ld", 99), ("k", -1), ("k", 1025), ("rows", 2 ** 60)):
            assert call(L, **{k: v}) == SHAPE, (k, v)
        for v in (0.0, -1.0, NAN, INF):
            assert call(L, scale=v) == VALUE
        for k in ("z", "i", "t"):
            assert call(L, **{k: None}) == NULL
        assert call(L, rows=0, z=None, i=None, t=None, g=None, loss=None, d=None, st=None) == OK
    for call in (dfwd, dboth):
        assert call(L, loss=None) == NULL and call(L, loss=X) == ALIAS and call(L, loss=W + 4) == ALIAS
        assert call(L, lse=Y) == ALIAS
    assert dfwd(L, st=Y) == ALIAS and dfwd(L, st=R) == ALIAS
    for call in (dbwd, dboth):
        assert call(L, g=None) == NULL and call(L, d=None) == NULL and call(L, ldo=99) == SHAPE
        assert call(L, d=X + 2) == ALIAS and call(L, d=X, ldo=108) == ALIAS and call(L, d=H) == ALIAS and call(L, d=R) == ALIAS
    assert dbwd(L, st=None) == NULL and dbwd(L, d=S) == ALIAS and dboth(L, d=Y) == ALIAS


def test_status():
    assert mfx.STATUS[9] == "MFX_ERR_VALUE"


def test_value_status_string(L):
    assert L.mfx_status_string(9) not in (b"unknown status", b"")


def test_binding_refuses():
    x, v, t = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: mfx.mfx_add_rmsnorm_fwd(x, v), lambda: mfx.mfx_add_rmsnorm_quant_fwd(x, v),
                 lambda: mfx.mfx_add_rmsnorm_bwd(x, x, v, v), lambda: mfx.mfx_token_logprobs_fwd(x, t),
                 lambda: mfx.mfx_token_logprobs_bwd(v, v, x, t, x),
                 lambda: mfx.mfx_topk_distill_fwd(x, t, x), lambda: mfx.mfx_topk_distill_fwd_bwd(x, t, x, v),
                 lambda: mfx.mfx_topk_distill_bwd(v, x, t, x, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    for call in (lambda: mfx.mfx_add_rmsnorm_fwd(x.half(), v), lambda: mfx.mfx_token_logprobs_fwd(x.half(), t)):
        with pytest.raises(TypeError):
            call()
