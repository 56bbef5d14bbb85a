"""Distillation of rows whose list holds nothing, with the teacher's own log of
its sum: loss 0 and a gradient of zeros whatever that log is, beside rows with
entries, in all three calls."""
import math

import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import distill, distill_bwd, excess, half

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
INF = math.inf
# exp(-lse) passes fp32's range from -88.7 down; -inf is what the log of a sum over nothing is
LSES = [-INF, torch.finfo(F32).min, -1000.0, -100.0, -88.8, -88.0, 0.0, 1000.0, INF, math.nan]


def rows_of(rows, vocab, k, dtype, teacher):
    """Logits, lists of which every second one holds nothing (no column, or
    only teacher logits of -inf), and the lse of each."""
    z = (torch.randn((rows, vocab), device=DEV) * 3).to(dtype)
    index = torch.randint(0, vocab, (rows, k), device=DEV)
    t = torch.randn((rows, k), device=DEV).to(teacher)
    lse = torch.logsumexp(t.float() * 0.7, 1) + 0.5 if k else torch.zeros(rows, device=DEV)
    n = torch.arange(rows, device=DEV)
    empty = (n % 2 == 0) | (k == 0)
    index[n % 4 == 0] = -1
    t[n % 4 == 2] = -INF
    lse = torch.where(empty, torch.tensor(LSES, device=DEV)[(n // 4) % len(LSES)], lse)
    return z, index, t, lse, empty


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab,k,teacher", [(44, 1000, 5, F32), (44, 131, 40, BF), (44, 1000, 0, F32), (1200, 700, 3, F32),
                                                  (44, 70001, 9, BF), (640, 20011, 33, F32), (44, 600007, 12, F32)])
def test_rows_without_entries(rows, vocab, k, teacher, dtype):
    z, index, t, lse, empty = rows_of(rows, vocab, k, dtype, teacher)
    g = torch.randn(rows, device=DEV)
    g[4], g[6], g[8] = 0.0, INF, 0.0  # a weight that says nothing, or too much, of a row that is left out
    kw = dict(scale=0.7, teacher_lse=lse)
    loss, stats = mfx.mfx_topk_distill_fwd(z, index, t, **kw)
    d = mfx.mfx_topk_distill_bwd(g, z, index, t, stats, **kw)
    loss2, d2 = mfx.mfx_topk_distill_fwd_bwd(z, index, t, g, **kw)
    assert loss[empty].eq(0).all() and loss2[empty].eq(0).all()
    assert d[empty].eq(0).all() and d2[empty].eq(0).all()
    on = ~empty
    if on.any():  # the other rows as ever
        r, q, want, tol, q_tol = distill(z[on], index[on], t[on], 0.7, lse[on])
        d_want, d_tol = distill_bwd(r, q, q_tol, index[on], g[on], 0.7, vocab)
        d_tol = d_tol + d_want.abs() * half(dtype)
        for a, b in ((loss, d), (loss2, d2)):
            assert excess(a[on], want, tol) <= 1 and excess(b[on], d_want, d_tol) <= 1


def test_in_place_and_nan():
    """The gradient over the logits; a teacher's NaN is no empty list."""
    z, index, t, lse, empty = rows_of(44, 5003, 6, BF, F32)
    t[1, 2] = math.nan
    g = torch.rand(44, device=DEV)
    loss, stats = mfx.mfx_topk_distill_fwd(z, index, t, teacher_lse=lse)
    d = mfx.mfx_topk_distill_bwd(g, z, index, t, stats)
    assert loss[1].isnan() and d[1].isnan().all() and d[empty].eq(0).all()
    for z2, call in ((z.clone(), lambda z2: mfx.mfx_topk_distill_bwd(g, z2, index, t, stats, dlogits=z2)),
                     (z.clone(), lambda z2: mfx.mfx_topk_distill_fwd_bwd(z2, index, t, g, teacher_lse=lse, dlogits=z2)[1])):
        call(z2)
        assert z2[empty].eq(0).all() and z2[1].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(44, 1000), (44, 131), (1200, 700), (44, 70001), (640, 20011), (44, 600007)])
def test_logits_of_rows_left_out_are_anything(rows, vocab, dtype):
    """A padded batch: rows without entries hold NaN and infinities."""
    z, index, t, _, _ = rows_of(rows, vocab, 5, dtype, F32)
    empty = torch.arange(rows, device=DEV) % 2 == 0
    g = torch.randn(rows, device=DEV)
    for lse in (None, torch.where(empty, -INF, torch.logsumexp(t, 1) + 0.5)):
        y = z.clone()
        y[0::8], y[2::8, 3], y[4::8, vocab // 2], y[6::8, -1] = math.nan, math.nan, INF, -INF
        loss, stats = mfx.mfx_topk_distill_fwd(y, index, t, teacher_lse=lse)
        d = mfx.mfx_topk_distill_bwd(g, y, index, t, stats)
        loss2, d2 = mfx.mfx_topk_distill_fwd_bwd(y, index, t, g, teacher_lse=lse)
        clean, d_clean = mfx.mfx_topk_distill_fwd_bwd(z, index, t, g, teacher_lse=lse)
        assert loss[empty].eq(0).all() and loss2[empty].eq(0).all()
        assert d[empty].eq(0).all() and d2[empty].eq(0).all()
        assert torch.equal(loss2[~empty], clean[~empty]) and torch.equal(d2[~empty], d_clean[~empty])
        mfx.mfx_topk_distill_fwd_bwd(y, index, t, g, teacher_lse=lse, dlogits=y)
        assert torch.equal(y, d2)
