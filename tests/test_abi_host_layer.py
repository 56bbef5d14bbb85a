"""Host-side refusals of the relative-position softmax, the dropouts without a
mask and the expert maps and copies (no GPU: every call below returns from
host validation), and the binding's own checks."""
import ctypes as C

import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from elementwise_epilogues_transformer_gb300 import build as B

OK, NULL, SHAPE, DTYPE, PROB, ALIAS, CUDA, DEVICE, WORKSPACE = range(9)

# Fake, never-dereferenced device addresses, far apart.
X, Y, Z, T, M, S, D, W_ = (0x100000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def L():
    B.build()
    return mfx.lib()


RELBIAS = dict(dt=1, b=2, np=4, sq=8, sk=16, scale=0.125, tdt=1, table=T, buckets=32, far=128, two=1, mask=None, mb=1,
               mnp=1, msq=1, causal=0, q=0, starts=None, p=0.1, seed=1, off=0, base=0)


def shared(a):
    return [a[k] for k in ("tdt", "table", "buckets", "far", "two", "mask", "mb", "mnp", "msq", "causal", "q",
                           "starts", "p", "seed", "off", "base")]


def forward(L, **k):
    a = {**RELBIAS, "x": X, "y": Y, "stats": S, **k}
    return L.mfx_relbias_softmax_dropout_fwd(a["dt"], a["b"], a["np"], a["sq"], a["sk"], a["x"], a["scale"],
                                             *shared(a), a["y"], a["stats"], None)


def backward(L, **k):
    a = {**RELBIAS, "x": X, "dy": Z, "stats": S, "dx": Y, "dtable": D, "ws": W_, "bytes": 1 << 20, **k}
    size = C.c_size_t(a["bytes"]) if a["bytes"] is not None else None
    st = L.mfx_relbias_softmax_dropout_bwd(a["dt"], a["b"], a["np"], a["sq"], a["sk"], a["dy"], a["x"], a["stats"],
                                           a["scale"], *shared(a), a["dx"], a["dtable"], a["ws"],
                                           C.byref(size) if size is not None else None, None)
    return (st, size.value) if size is not None else (st, None)


@pytest.mark.parametrize("call", [forward, lambda L, **k: backward(L, **k)[0]])
def test_relbias_sizes_and_types(L, call):
    assert call(L, dt=7) == DTYPE
    assert call(L, tdt=5) == DTYPE
    for p in (1.0, -0.1, float("nan")):
        assert call(L, p=p) == PROB
    for k in ("b", "np", "sq", "sk"):
        assert call(L, **{k: -1}) == SHAPE
        assert call(L, **{k: 2 ** 29 + 1}) == SHAPE
    assert call(L, b=2 ** 28, np=2 ** 28, sq=2 ** 28) == SHAPE
    assert call(L, q=2 ** 29 + 1) == SHAPE and call(L, q=-2 ** 29 - 1) == SHAPE
    assert call(L, base=2 ** 64 - 8) == SHAPE
    # masks that are neither broadcast nor x's size
    assert call(L, mask=M, mb=3) == SHAPE
    assert call(L, mask=M, mnp=2) == SHAPE
    assert call(L, mask=M, msq=16) == SHAPE
    # bucket functions
    for buckets, far, two in ((0, 128, 0), (1, 128, 0), (2, 128, 1), (31, 128, 1), (258, 2000, 1), (130, 2000, 0),
                              (32, 8, 1), (32, 16, 0), (32, 2049, 1), (-4, 128, 0)):
        assert call(L, buckets=buckets, far=far, two=two) == SHAPE, (buckets, far, two)


def test_relbias_pointers(L):
    for k in ("x", "y"):
        assert forward(L, **{k: None}) == NULL
    assert forward(L, b=0, x=None, y=None, stats=None) == OK
    n = 2 * 4 * 8 * 16 * 2  # bytes of x
    assert forward(L, y=X + 2) == ALIAS
    assert forward(L, y=T - n + 2) == ALIAS               # y over the table
    assert forward(L, mask=Y + 16) == ALIAS               # mask inside y
    assert forward(L, stats=X + n - 4) == ALIAS           # stats over x's end
    assert forward(L, stats=Y) == ALIAS
    assert forward(L, starts=Y + 4) == ALIAS
    for k in ("x", "dy", "stats", "dx"):
        assert backward(L, **{k: None})[0] == NULL
    assert backward(L, table=None)[0] == NULL             # a gradient without a table
    assert backward(L, bytes=None)[0] == NULL             # a gradient without a workspace
    assert backward(L, dx=X + 2)[0] == ALIAS
    assert backward(L, dx=Z - 4)[0] == ALIAS
    assert backward(L, dtable=Y + 8)[0] == ALIAS
    assert backward(L, dtable=T)[0] == ALIAS
    assert backward(L, ws=X)[0] == ALIAS
    assert backward(L, dtable=W_ + 16)[0] == ALIAS


def test_relbias_workspace(L):
    st, need = backward(L, ws=None, bytes=0)
    assert st == OK and need > 0 and need % (32 * 4 * 4) == 0
    assert backward(L, ws=None, bytes=0, x=None, dy=None, stats=None, dx=None, dtable=None) == (OK, need)
    assert backward(L, bytes=need - 1)[0] == WORKSPACE
    assert backward(L, ws=W_ + 8, bytes=need)[0] == WORKSPACE
    assert backward(L, ws=None, bytes=0, table=None, dtable=None) == (OK, 0)
    assert backward(L, ws=None, bytes=99, sk=0) == (OK, 0)


def test_dropout_validation(L):
    for name in ("mfx_dropout_fwd", "mfx_dropout_bwd"):
        f = getattr(L, name)
        assert f(3, 64, X, 0.1, 1, 0, 0, Y, None) == DTYPE
        assert f(1, -1, X, 0.1, 1, 0, 0, Y, None) == SHAPE
        assert f(1, 2 ** 62, X, 0.1, 1, 0, 0, Y, None) == SHAPE
        assert f(1, 64, X, 0.1, 1, 0, 2 ** 64 - 8, Y, None) == SHAPE
        assert f(1, 64, X, 1.0, 1, 0, 0, Y, None) == PROB
        assert f(1, 64, None, 0.1, 1, 0, 0, Y, None) == NULL
        assert f(1, 64, X, 0.1, 1, 0, 0, None, None) == NULL
        assert f(1, 64, X, 0.1, 1, 0, 0, X + 2, None) == ALIAS
        assert f(1, 0, None, 0.1, 1, 0, 0, None, None) == OK
    f = L.mfx_bias_dropout_add_train_nomask
    assert f(1, 9, 4, 8, X, None, Y, 0.1, 1, 0, 0, Z, None) == DTYPE
    assert f(1, 0, 4, 8, X, None, Y, float("nan"), 1, 0, 0, Z, None) == PROB
    assert f(1, 0, -4, 8, X, None, Y, 0.1, 1, 0, 0, Z, None) == SHAPE
    assert f(1, 0, 4, 8, X, None, Y, 0.1, 1, 0, 2 ** 64 - 4, Z, None) == SHAPE
    for args in ((None, Y, Z), (X, None, Z), (X, Y, None)):
        assert f(1, 0, 4, 8, args[0], None, args[1], 0.1, 1, 0, 0, args[2], None) == NULL
    assert f(1, 0, 4, 8, X, None, Y, 0.1, 1, 0, 0, X + 2, None) == ALIAS
    assert f(1, 0, 4, 8, X, None, Y, 0.1, 1, 0, 0, Y, None) == ALIAS
    assert f(1, 0, 4, 8, X, Z + 2, Y, 0.1, 1, 0, 0, Z, None) == ALIAS
    assert f(1, 0, 0, 8, None, None, None, 0.1, 1, 0, 0, None, None) == OK


def sort(L, ws=W_, size=1 << 20, **k):
    a = dict(tokens=8, topk=2, experts=4, align=1, capacity=0, rows=16, e=X, r=Y, s=Z, o=T, c=M)
    a.update(k)
    n = C.c_size_t(size)
    st = L.mfx_moe_sort(a["tokens"], a["topk"], a["experts"], a["align"], a["capacity"], a["rows"], a["e"], a["r"],
                        a["s"], a["o"], a["c"], ws, C.byref(n), None)
    return st, n.value


def test_sort_validation(L):
    for k, v in (("tokens", -1), ("topk", -1), ("experts", 0), ("experts", 4097), ("align", 0), ("capacity", -1),
                 ("rows", 15), ("rows", -1), ("rows", 2 ** 31), ("tokens", 2 ** 31), ("align", 2 ** 31)):
        assert sort(L, **{k: v})[0] == SHAPE, (k, v)
    assert sort(L, align=16)[0] == SHAPE                      # rows for packed experts only
    assert sort(L, ws=None, align=16, rows=76) == (OK, 0)
    assert sort(L, ws=None, align=16, rows=75)[0] == SHAPE
    assert sort(L, ws=None, capacity=3, rows=12) == (OK, 0)   # what the capacity allows
    assert sort(L, ws=None, capacity=3, rows=11)[0] == SHAPE
    for k in ("e", "r", "s", "o", "c"):
        assert sort(L, **{k: None})[0] == NULL
    assert sort(L, r=X)[0] == ALIAS and sort(L, s=Y + 60)[0] == ALIAS and sort(L, o=M)[0] == ALIAS
    st, need = sort(L, ws=None, tokens=5000, rows=10000)
    assert st == OK and need == 5 * 4 * 4                     # five blocks' counts
    assert sort(L, size=need - 1, tokens=5000, rows=10000)[0] == WORKSPACE
    assert sort(L, ws=W_ + 4, tokens=5000, rows=10000)[0] == WORKSPACE
    assert L.mfx_moe_sort(8, 2, 4, 1, 0, 16, X, Y, Z, T, M, W_, None, None) == NULL


def test_sort_without_workspace(L):
    """Both null where the size is 0 (checked on a GPU), an error where it is not."""
    assert L.mfx_moe_sort(5000, 2, 4, 1, 0, 10000, X, Y, Z, T, M, None, None, None) == NULL
    assert L.mfx_moe_sort(8, 2, 4, 1, 0, 16, X, None, Z, T, M, None, None, None) == NULL
    assert L.mfx_moe_sort(8, 2, 4, 1, 0, 16, X, X, Z, T, M, None, None, None) == ALIAS


def test_rows():
    assert mfx.mfx_moe_rows(10, 2, 4, 1) == 20
    assert mfx.mfx_moe_rows(10, 2, 4, 16) == 20 + 4 * 15
    assert mfx.mfx_moe_rows(1, 2, 64, 16) == 2 + 2 * 15       # no more experts than slots
    assert mfx.mfx_moe_rows(0, 2, 4, 16) == 0
    for bad in ((-1, 2, 4, 1), (1, 2, 4, 0), (2 ** 40, 2 ** 40, 4, 1)):
        with pytest.raises(mfx.MfxError):
            mfx.mfx_moe_rows(*bad)


def test_copy_validation(L):
    p, pb, u, ub = (L.mfx_moe_permute_fwd, L.mfx_moe_permute_bwd, L.mfx_moe_unpermute_fwd, L.mfx_moe_unpermute_bwd)
    assert p(4, 8, 2, 16, 16, X, T, M, None, Y, None, None) == DTYPE
    for bad in ((-1, 2, 16, 16), (8, -2, 16, 16), (8, 2, -16, 16), (8, 2, 16, -16), (8, 2, 16, 2 ** 31),
                (2 ** 40, 2 ** 40, 16, 16), (2 ** 30, 1, 2 ** 40, 16)):
        assert p(1, *bad, X, T, M, None, Y, None, None) == SHAPE
        assert pb(1, *bad, X, T, None, Y, None, None) == SHAPE
        assert u(1, *bad, X, T, None, Y, None) == SHAPE
        assert ub(1, *bad, X, Z, T, M, None, Y, None, None) == SHAPE
    z = (1, 8, 2, 16, 16)
    assert p(*z, None, T, M, None, Y, None, None) == NULL and p(*z, X, None, M, None, Y, None, None) == NULL
    assert p(*z, X, T, None, None, Y, None, None) == NULL and p(*z, X, T, M, None, None, None, None) == NULL
    assert p(*z, X, T, M, S, Y, None, None) == NULL           # weights without a place for them
    assert p(*z, X, T, M, None, Y, D, None) == NULL           # and the reverse
    assert p(*z, X, T, M, None, X + 16, None, None) == ALIAS and p(*z, X, T, M, S, Y, Y + 4, None) == ALIAS
    assert p(*z, X, Y + 4, M, None, Y, None, None) == ALIAS
    assert pb(*z, None, T, None, Y, None, None) == NULL and pb(*z, X, T, S, Y, None, None) == NULL
    assert pb(*z, X, T, None, Y, D, None) == NULL and pb(*z, X, T, None, X, None, None) == ALIAS
    assert u(*z, X, None, None, Y, None) == NULL and u(*z, X, T, None, None, None) == NULL
    assert u(*z, X, T, Y + 8, Y, None) == ALIAS
    assert ub(*z, X, None, T, M, S, Y, D, None) == NULL       # dweight without y
    assert ub(*z, None, Z, T, M, S, Y, D, None) == NULL and ub(*z, X, Z, T, None, S, Y, D, None) == NULL
    assert ub(*z, X, Z, T, M, S, Z, D, None) == ALIAS and ub(*z, X, Z, T, M, S, Y, Y + 4, None) == ALIAS
    assert ub(*z, X, Z, T, M, S, Y, S, None) == ALIAS
    for empty in ((1, 8, 2, 0, 16), (1, 0, 2, 16, 0)):
        assert p(*empty, None, None, None, None, None, None, None) == OK
        assert pb(*empty, None, None, None, None, None, None) == OK
        assert u(*empty, None, None, None, None, None) == OK
        assert ub(*empty, None, None, None, None, None, None, None, None) == OK


def test_copies_without_columns_need_their_maps(L):
    """Width 0 with weights is work still to be done, so what it reads and writes has to be there."""
    p, pb, ub = L.mfx_moe_permute_fwd, L.mfx_moe_permute_bwd, L.mfx_moe_unpermute_bwd
    z = (1, 8, 2, 0, 16)
    assert p(*z, None, T, None, S, None, D, None) == NULL and p(*z, None, None, M, S, None, D, None) == NULL
    assert p(*z, None, T, M, S, None, None, None) == NULL and p(*z, None, T, M, None, None, D, None) == NULL
    assert p(*z, None, T, M, S, None, S, None) == ALIAS and p(*z, None, T, M, S, None, M + 4, None) == ALIAS
    assert pb(*z, None, None, S, None, D, None) == NULL and pb(*z, None, T, S, None, None, None) == NULL
    assert pb(*z, None, T, None, None, D, None) == NULL
    assert pb(*z, None, T, S, None, S + 4, None) == ALIAS
    assert ub(*z, None, None, None, None, S, None, None, None) == OK


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(2, 4, 8, 16)
    for call in (lambda: mfx.mfx_relbias_softmax_dropout_fwd(x, 1.0),
                 lambda: mfx.mfx_dropout_fwd(x, 0.1, 1),
                 lambda: mfx.mfx_bias_dropout_add_train_nomask(x, None, x, 0.1, 1),
                 lambda: mfx.mfx_moe_sort(torch.zeros(4, 2, dtype=torch.int32), 3),
                 lambda: mfx.mfx_moe_unpermute_fwd(x[0, 0], torch.zeros(8, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_workspace_sizes_kept_are_bounded(monkeypatch):
    """Calls of ever new sizes do not make the binding grow; sizes seen lately are not asked for again."""
    asked = []
    monkeypatch.setattr(mfx, "_workspace_bytes", {})
    monkeypatch.setattr(mfx, "_call", lambda name, *args: asked.append(args[0]) if args[-2] is not None else None)
    sort = lambda n: mfx._with_workspace("mfx_moe_sort", (n,), (0,), None, sizes=(n, 8), none=True)
    for n in range(5000):
        sort(n)
        sort(n)
    assert asked == list(range(5000))
    assert 0 < len(mfx._workspace_bytes) <= 1024
