"""The norm with the residual's addition against 64 bits: every layout of a
row, types, 8-bit outputs, misaligned buffers, in place, long rows, gradients."""
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import U, excess, half, norm_bwd, norm_fwd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
DEV = "cuda:0"

# widths on both sides of every change of layout (8 lanes to a block, one to four runs a thread, longer rows)
WIDTHS = [1, 7, 8, 64, 65, 72, 128, 136, 250, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2051, 2056, 4096, 5003, 8192,
          8200, 16384, 16392, 20001, 32768, 32776]


def rand(shape, dtype, std=1.0):
    return (torch.randn(shape, device=DEV) * std).to(dtype)


def off_by_one(t):
    """The same values an element off a vector."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


def check_fwd(x, residual, weight, eps=1e-6, offset=0.0, **kw):
    y, h, rstd = mfx.mfx_add_rmsnorm_fwd(x, weight, residual=residual, eps=eps, weight_offset=offset, **kw)
    h32, want, r, rel = norm_fwd(x, residual, weight, eps, offset)
    assert excess(y, want, want.abs() * (half(y.dtype) + rel)) <= 1
    assert excess(rstd.view(r.shape), r, r.abs() * rel) <= 1
    if residual is None:
        assert h is None
    else:
        assert torch.equal(h, h32.to(residual.dtype))
    return y, h, rstd


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("xdt,rdt", [(BF, None), (BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_fwd(cols, xdt, rdt):
    for rows in (1, 5, 37):
        x = rand((rows, cols), xdt)
        residual = None if rdt is None else rand((rows, cols), rdt, 3.0)
        check_fwd(x, residual, rand((cols,), xdt, 0.3) + 1)


@pytest.mark.parametrize("cols", [64, 1000, 2051, 4096, 40000])
def test_many_rows(cols):
    rows = 20000 if cols <= 4096 else 700
    check_fwd(rand((rows, cols), BF), rand((rows, cols), F32), rand((cols,), F32), offset=1.0)


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("cols", [64, 1024, 4096])
def test_misaligned(cols, which):
    x, residual, weight = rand((9, cols), BF), rand((9, cols), F32), rand((cols,), BF)
    t = [x, residual, weight]
    if which < 3:
        t[which] = off_by_one(t[which])
        check_fwd(*t)
    else:
        y = off_by_one(torch.empty_like(x))
        check_fwd(*t, y=y)


def test_shapes_weights_and_extremes():
    x = rand((3, 4, 96), BF)
    check_fwd(x, rand((3, 4, 96), BF), None)
    check_fwd(x, None, rand((96,), F32), offset=1.0)
    # rows of zeros, tiny and large values, infinities and NaN
    x = torch.stack([torch.zeros(512), torch.full((512,), 1e-20), torch.full((512,), 1e15)]).to(DEV)
    check_fwd(x, None, rand((512,), F32))
    x = rand((3, 512), F32)
    x[0, 3], x[1, 5] = float("nan"), float("inf")
    y, _, _ = mfx.mfx_add_rmsnorm_fwd(x, None)
    assert y[0].isnan().all() and y[1, 5].isnan() and (y[1, :5] == 0).all() and y[2].isfinite().all()
    for shape in ((0, 512), (4, 0)):
        y, h, rstd = mfx.mfx_add_rmsnorm_fwd(rand(shape, BF), rand(shape[1:], BF), residual=rand(shape, F32))
        assert y.shape == shape and h.shape == shape


@pytest.mark.parametrize("cols", [72, 1024, 2051, 4096, 33000])
def test_in_place(cols):
    x, residual, weight = rand((50, cols), BF), rand((50, cols), F32), rand((cols,), BF)
    y, h, _ = mfx.mfx_add_rmsnorm_fwd(x, weight, residual=residual)
    x2, r2 = x.clone(), residual.clone()
    y2, h2, _ = mfx.mfx_add_rmsnorm_fwd(x2, weight, residual=r2, y=x2, h=r2)
    assert torch.equal(y, x2) and torch.equal(h, r2)


def dequantised(q, scale, group):
    cols = q.shape[-1]
    return q.double() * scale.double().repeat_interleave(group or cols, -1)[..., :cols]


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("qdt,sdt", [(E4, F32), (E4, E8), (E5, F32), (E5, E8)])
@pytest.mark.parametrize("cols", WIDTHS + [40000])
def test_quant(cols, qdt, sdt, group):
    x, residual, weight = rand((11, cols), BF), rand((11, cols), F32, 2.0), rand((cols,), F32)
    x[3], residual[3] = 0, 0
    weight[:min(cols, 40)] *= 1e-3  # a small group
    q, scale, h, rstd = mfx.mfx_add_rmsnorm_quant_fwd(x, weight, residual=residual, group=group, q_dtype=qdt,
                                                      scale_dtype=sdt, need_rstd=True)
    h32, y, r, rel = norm_fwd(x, residual, weight, 1e-6, 0.0)
    assert torch.equal(h, h32) and excess(rstd, r, r * rel) <= 1
    most = torch.finfo(qdt).max
    n = group or cols
    tops = torch.stack([p.abs().max(1).values for p in y.split(n, 1)], 1)
    ideal = torch.where(tops == 0, 1.0, (tops / most).clamp(min=2.0 ** -126))
    if sdt is E8:
        s = scale.double()
        assert ((s == 1) | (ideal != 1))[3].all()
        # the power of two next above, either one where the largest value lies on a power's border
        assert (s * (1 + 3 * rel) >= ideal).all() and (s < 2 * ideal * (1 + 3 * rel))[ideal != 1].all()
    else:
        assert excess(scale, ideal, ideal * (rel + 4 * U)) <= 1
    # half a step of the type, or of its smallest numbers
    step, least = torch.finfo(qdt).eps / 2, torch.finfo(qdt).smallest_normal * torch.finfo(qdt).eps / 2
    s = scale.double().repeat_interleave(n, 1)[:, :cols]
    assert excess(dequantised(q, scale, group), y, y.abs() * (step + 2 * rel + 8 * U) + s * least * (1 + 1e-6)) <= 1


def test_quant_rounding_and_specials():
    # a group's largest value is the type's largest
    x = torch.tensor([[448.0, 17.0, 19.0, -21.0] * 8], device=DEV)
    x = torch.cat([x, x], 1)
    q, s, _, _ = mfx.mfx_add_rmsnorm_quant_fwd(x, None, eps=0.0, group=32)
    y = x.double() / x.double().square().mean().sqrt()
    assert excess(dequantised(q, s, 32), y, y.abs() * (2.0 ** -4 + 1e-5)) <= 1
    assert q.float()[0, 0] == 448
    # NaN stays, an infinite row's finite elements are zero
    x = rand((2, 256), F32)
    x[0, 9] = float("nan")
    q, s, _, _ = mfx.mfx_add_rmsnorm_quant_fwd(x, None, group=128)
    assert q.float()[0].isnan().all() and (s[0] == 1).all() and q.float()[1].isfinite().all()
    # weights so large that y overflows: saturated
    w = torch.full((256,), 3e38, device=DEV)
    x = torch.ones((1, 256), device=DEV)
    x[0, :4] = 100.0
    q, s, _, _ = mfx.mfx_add_rmsnorm_quant_fwd(x, w, group=0)
    assert (q.float()[0, :4] == 448).all() and s.isfinite().all()
    for shape in ((0, 512), (4, 0)):
        q, s, h, _ = mfx.mfx_add_rmsnorm_quant_fwd(rand(shape, BF), None, group=32)
        assert q.shape == shape and s.numel() == 0
    # q an element off 8 bytes
    x, w = rand((5, 512), BF), rand((512,), BF)
    q, s, _, _ = mfx.mfx_add_rmsnorm_quant_fwd(x, w, group=128)
    q2 = torch.empty(5 * 512 + 1, dtype=E4, device=DEV)[1:].view(5, 512)
    _, s2, _, _ = mfx.mfx_add_rmsnorm_quant_fwd(x, w, group=128, q=q2)
    y = norm_fwd(x, None, w, 1e-6, 0.0)[1]
    assert excess(dequantised(q2, s2, 128), y, y.abs() * (2.0 ** -4 + 1e-5) + s2.double().repeat_interleave(128, 1) * 2.0 ** -10 * 1.0001) <= 1


def check_bwd(dy, h, rstd, weight, dh=None, offset=0.0, **kw):
    res = h.dtype
    dx, dres, dw = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, weight, dh=dh, weight_offset=offset, residual_dtype=res, **kw)
    d, tol, w, w_tol = norm_bwd(dy, h, rstd, weight, dh, offset)
    assert excess(dx, d, tol + d.abs() * half(dx.dtype)) <= 1
    assert excess(dres, d, tol + d.abs() * half(res)) <= 1
    if weight is None:
        assert dw is None
    else:
        assert excess(dw, w, w_tol + w.abs() * half(dw.dtype)) <= 1
    return dx, dres, dw


@pytest.mark.parametrize("cols", WIDTHS + [40000])
@pytest.mark.parametrize("xdt,rdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_bwd(cols, xdt, rdt):
    for rows in (1, 37):
        h, dy, dh = rand((rows, cols), rdt, 2.0), rand((rows, cols), xdt), rand((rows, cols), rdt)
        rstd = 1.0 / torch.sqrt(h.float().square().mean(1) + 1e-6)
        check_bwd(dy, h, rstd, rand((cols,), xdt) + 1, dh)
        check_bwd(dy, h, rstd, rand((cols,), F32), None, 1.0)


@pytest.mark.parametrize("cols", [64, 520, 1000, 2051, 4096, 8192, 33000])
def test_bwd_many_rows(cols):
    rows = 9000 if cols <= 8192 else 800
    h, dy, dh = rand((rows, cols), F32, 2.0), rand((rows, cols), BF), rand((rows, cols), F32)
    rstd = 1.0 / torch.sqrt(h.square().mean(1) + 1e-6)
    w = rand((cols,), BF)
    a = check_bwd(dy, h, rstd, w, dh)
    b = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, w, dh=dh, residual_dtype=F32)
    assert all(torch.equal(p, q) for p, q in zip(a, b))  # the same bits again
    dx, dres, dw = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, w, dh=dh, need_dweight=False)
    assert torch.equal(dx, a[0]) and dres is None and dw is None


@pytest.mark.parametrize("cols", [128, 1024, 4096, 33000])
def test_bwd_in_place_and_misaligned(cols):
    h, dy, dh, w = rand((21, cols), F32), rand((21, cols), BF), rand((21, cols), F32), rand((cols,), BF)
    rstd = 1.0 / torch.sqrt(h.square().mean(1) + 1e-6)
    dx, dres, dw = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, w, dh=dh, residual_dtype=F32)
    a, b = dy.clone(), dh.clone()
    _, _, dw2 = mfx.mfx_add_rmsnorm_bwd(a, h, rstd, w, dh=b, dx=a, dresidual=b)
    assert torch.equal(a, dx) and torch.equal(b, dres) and torch.equal(dw, dw2)
    for which in range(4):
        t = [dy, h, w, dh]
        t[which] = off_by_one(t[which])
        check_bwd(t[0], t[1], rstd, t[2], t[3])
    check_bwd(dy, h, rstd, w, dh, dx=off_by_one(torch.empty_like(dy)))
    check_bwd(dy, h, rstd, w, dh, dresidual=off_by_one(torch.empty_like(h)))


def test_bwd_empty():
    w = rand((512,), BF)
    dx, _, dw = mfx.mfx_add_rmsnorm_bwd(rand((0, 512), BF), rand((0, 512), BF), rand((0,), F32), w)
    assert dx.shape == (0, 512) and (dw == 0).all()
    dx, _, dw = mfx.mfx_add_rmsnorm_bwd(rand((4, 0), BF), rand((4, 0), BF), rand((4,), F32), rand((0,), BF))
    assert dx.shape == (4, 0) and dw.shape == (0,)


def test_bwd_against_differences():
    """The gradients against differences of the 64-bit loss along random directions."""
    rows, cols = 6, 264
    x, res, w, dy, dh = (rand(s, F32) for s in ((rows, cols), (rows, cols), (cols,), (rows, cols), (rows, cols)))
    _, h, rstd = mfx.mfx_add_rmsnorm_fwd(x, w, residual=res)
    dx, dres, dw = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, w, dh=dh, residual_dtype=F32)

    def loss(x, w):
        hh = x.double() + res.double()
        y = hh / torch.sqrt(hh.square().mean(1, keepdim=True) + 1e-6) * w.double()
        return (y * dy.double()).sum() + (hh * dh.double()).sum()

    vx, vw = torch.randn_like(x).double(), torch.randn_like(w).double()
    s = 1e-5
    by_x = (loss(x.double() + s * vx, w) - loss(x.double() - s * vx, w)) / (2 * s)
    by_w = (loss(x, w.double() + s * vw) - loss(x, w.double() - s * vw)) / (2 * s)
    # 32-bit gradients: 2^-24 a term of sums of 6 * 264; differences: s^2 of third derivatives of order one
    size = (dx.double() * vx).abs().sum()
    assert abs((dx.double() * vx).sum() - by_x) <= 1e-6 * size
    assert abs((dw.double() * vw).sum() - by_w) <= 1e-6 * (dw.double() * vw).abs().sum()
    assert torch.equal(dx, dres)


@pytest.mark.parametrize("cols", [264, 504, 512, 520, 768, 1000, 1024, 1032, 1544, 2048, 2056, 4096, 5000, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_of_one_type(cols, dtype):
    """Up to 32 elements a thread, with rows on their way: forward, in place,
    8 bits with a scale a row, backward in place, the same bits again."""
    rows = 1203
    x, residual, weight = rand((rows, cols), dtype), rand((rows, cols), dtype, 2.0), rand((cols,), dtype, 0.3) + 1
    y, h, rstd = check_fwd(x, residual, weight)
    x2, r2 = x.clone(), residual.clone()
    mfx.mfx_add_rmsnorm_fwd(x2, weight, residual=r2, y=x2, h=r2)
    assert torch.equal(y, x2) and torch.equal(h, r2)
    q, scale, h2, _ = mfx.mfx_add_rmsnorm_quant_fwd(x, weight, residual=residual)
    assert torch.equal(h, h2)
    want, _, rel = norm_fwd(x, residual, weight, 1e-6, 0.0)[1:]
    # half a step of the type, or of its smallest numbers
    assert excess(dequantised(q, scale, 0), want, want.abs() * (2.0 ** -4 + 2 * rel + 8 * U) + scale.double().view(-1, 1) * 2.0 ** -10 * (1 + 1e-6)) <= 1
    dy, dh = rand((rows, cols), dtype), rand((rows, cols), dtype)
    a = check_bwd(dy, h, rstd, weight, dh)
    g = dy.clone()
    dx, _, dw = mfx.mfx_add_rmsnorm_bwd(g, h, rstd, weight, dh=dh, dx=g)
    assert torch.equal(dx, a[0]) and torch.equal(dw, a[2])
