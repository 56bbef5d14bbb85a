"""Token log probabilities and distillation against 64 bits: vocabulary sizes
around every change of layout, types, padded and misaligned rows, masks, ties,
few and many rows, gradients."""
import math

import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import distill, distill_bwd, excess, half, logprobs, logprobs_bwd, top_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
INF = math.inf
VOCABS = [1, 2, 7, 8, 9, 63, 64, 100, 257, 1000, 1024, 4099, 8192, 32003, 65536, 131072]


def logits_of(rows, vocab, dtype, pad=0, lead=0, std=3.0):
    """Rows `vocab + pad` apart that begin `lead` elements off their buffer."""
    flat = torch.randn(rows * (vocab + pad) + lead, device=DEV) * std
    z = flat.to(dtype)[lead:].view(rows, vocab + pad)
    if pad:
        z[:, vocab:] = float("nan")  # what lies between is not read
    return z[:, :vocab]


def tokens_of(rows, vocab, dtype=torch.int64, lost=True):
    t = torch.randint(0, vocab, (rows,), device=DEV)
    if lost and rows > 4:
        t[1], t[3] = -100, vocab
    return t.to(dtype)


def check(z, tokens, scale=1.0, top=0, g=None, ge=None, dlogits=None):
    rows, vocab = z.shape
    lp, ent, tv, ti, stats = mfx.mfx_token_logprobs_fwd(z, tokens, scale=scale, top=top)
    r, kept, want, tol = logprobs(z, tokens, scale)
    assert excess(lp, want, torch.where(kept, tol, 0.0)) <= 1
    assert excess(ent, torch.where(kept, r.entropy, 0.0), torch.where(kept, r.entropy_tol, 0.0)) <= 1
    if top:
        index = top_of(z, kept, top)
        assert torch.equal(ti.long(), index)
        at = index.clamp(min=0)
        want = torch.where(index < 0, -INF, r.logp.gather(1, at))
        assert excess(tv, want, torch.where(index < 0, 0.0, r.logp_tol.gather(1, at))) <= 1
    g = torch.randn(rows, device=DEV) if g is None else g
    ge = torch.randn(rows, device=DEV) if ge is None else ge
    for one, two in ((g, ge), (g, None), (None, ge)):
        d = mfx.mfx_token_logprobs_bwd(one, two, z, tokens, stats, scale=scale, dlogits=dlogits)
        want, tol = logprobs_bwd(r, kept, tokens, one, two, scale)
        assert excess(d, want, tol + want.abs() * half(z.dtype)) <= 1
    return lp, ent, tv, ti, stats


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logprobs(vocab, dtype):
    for rows, top in ((1, 5), (7, 64), (400 if vocab < 60000 else 160, 20)):
        check(logits_of(rows, vocab, dtype), tokens_of(rows, vocab), 0.7, top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,lead", [(1, 0), (3, 1), (8, 5), (0, 3), (13, 7)])
def test_logprobs_rows_apart(dtype, pad, lead):
    for vocab in (5, 1000, 4099, 70001):
        z = logits_of(9, vocab, dtype, pad, lead)
        check(z, tokens_of(9, vocab, torch.int32), 1.3, 3)
        # the gradient in rows of its own distance, what lies between left alone
        out = torch.full((9, vocab + 5), 7.0, dtype=dtype, device=DEV)
        check(z, tokens_of(9, vocab), 1.0, 0, dlogits=out[:, :vocab])
        assert (out[:, vocab:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [300, 5000, 66000])
def test_logprobs_masks(dtype, vocab):
    z = logits_of(8, vocab, dtype)
    z[0] = -INF                                  # nothing left
    z[1] = -INF
    z[1, vocab // 3] = 2.0                       # one column
    z[2, ::2] = -INF
    z[3] = torch.finfo(dtype).min                # the lowest value everywhere
    z[4, 5:] = torch.finfo(dtype).min
    z[5] = 0.0                                   # all equal
    z[6] = torch.finfo(dtype).max / 4
    z[7, :] = -INF
    z[7, -3:] = torch.tensor([1.0, -0.0, 0.0], dtype=dtype)
    t = torch.tensor([0, vocab // 3, 1, 2, 0, 9, 3, vocab - 1], device=DEV)
    lp, ent, tv, ti, stats = check(z, t, 0.5, 10)
    assert lp[0] == -INF and ent[0] == 0 and lp[1] == 0 and ent[1] == 0
    assert ti[5].tolist() == list(range(10)) and ti[1].tolist() == [vocab // 3] + [-1] * 9
    assert ti[7].tolist()[:3] == [vocab - 3, vocab - 2, vocab - 1]  # -0 and 0 are equal
    for scale in (1.0, 3.0):
        check(z, t, scale, 64)


@pytest.mark.parametrize("vocab", [300, 66000])
def test_logprobs_nan_and_inf(vocab):
    z = logits_of(4, vocab, F32)
    z[0, 17], z[1, 100], z[2, 3] = float("nan"), INF, float("nan")
    t = torch.tensor([2, 2, -1, 2], device=DEV)
    lp, ent, tv, ti, stats = mfx.mfx_token_logprobs_fwd(z, t, top=4)
    assert lp[:2].isnan().all() and ent[:2].isnan().all() and lp[2] == 0 and lp[3].isfinite()
    assert 17 not in ti[0].tolist() and ti[1, 0] == 100 and (ti[2] == -1).all()
    d = mfx.mfx_token_logprobs_bwd(torch.ones(4, device=DEV), None, z, t, stats)
    assert d[:2].isnan().all() and (d[2] == 0).all() and d[3].isfinite().all()


def test_top_ties_and_orders():
    """Ties, sorted rows, and rows whose large logits all belong to a few threads."""
    for vocab in (5000, 40000, 131072):
        rise = torch.arange(vocab, device=DEV, dtype=F32)
        few = torch.where((torch.arange(vocab, device=DEV) % 4096) < 8, 100.0, 0.0) + torch.rand(vocab, device=DEV)
        comb = torch.where((torch.arange(vocab, device=DEV) % 512) < 16, rise, -rise)
        ties = torch.randint(0, 3, (vocab,), device=DEV).float()
        one = torch.full((vocab,), -INF, device=DEV)
        one[torch.arange(0, vocab, 4096)] = 1.0
        z = torch.stack([rise, -rise, few, comb, ties, one])
        for rows in (z, z.repeat(60, 1)):
            for top in (1, 2, 20, 63, 64):
                t = torch.zeros(rows.shape[0], dtype=torch.int64, device=DEV)
                ti = mfx.mfx_token_logprobs_fwd(rows, t, top=top, need_stats=False)[3]
                assert torch.equal(ti.long(), top_of(rows, t >= 0, top))
    z = torch.randint(-2, 3, (50, 70000), device=DEV).to(BF)
    t = torch.zeros(50, dtype=torch.int32, device=DEV)
    assert torch.equal(mfx.mfx_token_logprobs_fwd(z, t, top=64)[3].long(), top_of(z, t >= 0, 64))


def test_logprobs_far_from_zero_and_peaked():
    z = logits_of(6, 3000, F32, std=1.0)
    z[:3] += 30000.0
    z[3, 7] += 40.0
    z[4] *= 1e30
    t = torch.tensor([1, 2, 3, 7, 5, 6], device=DEV)
    check(z, t, 1.0, 5)


def test_logprobs_in_place_and_large_rows():
    z = logits_of(33, 5003, BF)
    t = tokens_of(33, 5003)
    stats = mfx.mfx_token_logprobs_fwd(z, t)[4]
    g, ge = torch.randn(33, device=DEV), torch.randn(33, device=DEV)
    want = mfx.mfx_token_logprobs_bwd(g, ge, z, t, stats)
    got = mfx.mfx_token_logprobs_bwd(g, ge, z, t, stats, dlogits=z)
    assert got is z and torch.equal(z, want)
    big = logits_of(2, 1_000_003, F32)
    check(big, torch.tensor([999_999, 1_000_002], device=DEV), 1.0, 30)
    many = logits_of(40000, 130, BF)
    check(many, tokens_of(40000, 130), 1.0, 2)


def test_logprobs_empty():
    z = torch.empty((0, 100), device=DEV)
    lp, ent, tv, ti, st = mfx.mfx_token_logprobs_fwd(z, torch.empty(0, dtype=torch.int64, device=DEV), top=3)
    assert lp.shape == (0,) and tv.shape == (0, 3)
    z, t = torch.empty((3, 0), device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    lp, ent, tv, ti, st = mfx.mfx_token_logprobs_fwd(z, t, top=3)
    assert (lp == 0).all() and (ent == 0).all() and (ti == -1).all()
    assert mfx.mfx_token_logprobs_bwd(lp, ent, z, t, st).shape == (3, 0)


# --- distillation -----------------------------------------------------------
def lists_of(rows, vocab, k, index_dtype=torch.int64, teacher=F32, twice=False):
    index = torch.rand((rows, vocab), device=DEV).topk(min(k, vocab), 1).indices if not twice else None
    if index is None or index.shape[1] < k:
        index = torch.randint(0, vocab, (rows, k), device=DEV)
    if rows > 4 and k:
        index[1] = -1
        index[2, k // 2:] = -1
        index[3, 0] = vocab
    return index.to(index_dtype), (torch.randn((rows, k), device=DEV) * 3).to(teacher)


def check_distill(z, index, t, scale=1.0, lse=None, dlogits=None):
    rows, vocab = z.shape
    r, q, want, tol, q_tol = distill(z, index, t, scale, lse)
    loss, stats = mfx.mfx_topk_distill_fwd(z, index, t, scale=scale, teacher_lse=lse)
    assert excess(loss, want, tol) <= 1
    g = torch.randn(rows, device=DEV)
    d_want, d_tol = distill_bwd(r, q, q_tol, index, g, scale, vocab)
    d_tol = d_tol + d_want.abs() * half(z.dtype)
    d = mfx.mfx_topk_distill_bwd(g, z, index, t, stats, scale=scale, teacher_lse=lse, dlogits=dlogits)
    assert excess(d, d_want, d_tol) <= 1
    loss2, d2 = mfx.mfx_topk_distill_fwd_bwd(z, index, t, g, scale=scale, teacher_lse=lse, dlogits=dlogits)
    assert excess(loss2, want, tol) <= 1 and excess(d2, d_want, d_tol) <= 1
    return loss, d2


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_distill(vocab, dtype):
    for rows, k in ((1, 1), (7, 16), (300 if vocab < 60000 else 160, 64)):
        index, t = lists_of(rows, vocab, k, teacher=BF if rows == 7 else F32)
        check_distill(logits_of(rows, vocab, dtype), index, t, 0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,lead", [(1, 0), (8, 5), (13, 7)])
def test_distill_rows_apart(dtype, pad, lead):
    for vocab in (5, 1000, 70001):
        z = logits_of(9, vocab, dtype, pad, lead)
        index, t = lists_of(9, vocab, 12, torch.int32, twice=True)
        out = torch.full((9, vocab + 5), 7.0, dtype=dtype, device=DEV)
        lse = torch.logsumexp(t, 1) + 0.3
        check_distill(z, index, t, 1.0, lse, dlogits=out[:, :vocab])
        assert (out[:, vocab:] == 7).all()


@pytest.mark.parametrize("k", [1, 2, 33, 600, 1024])
@pytest.mark.parametrize("vocab", [40, 9000, 66000])
def test_distill_same_column_twice(k, vocab):
    index, t = lists_of(6, vocab, k, twice=True)
    index[0] = 3  # one column many times
    check_distill(logits_of(6, vocab, F32), index, t, 0.8)
    check_distill(logits_of(6, vocab, BF), index, t, 1.0, torch.logsumexp(t, 1) + 1)


def test_distill_masks_and_specials():
    vocab = 5000
    z = logits_of(8, vocab, F32)
    index, t = lists_of(8, vocab, 8)
    index = index.clamp(min=0) % vocab
    z[0] = -INF                       # no student left
    z[1, index[1, 2]] = -INF          # the teacher likes a column that is ruled out
    z[2] = torch.finfo(F32).min
    t[3] = -INF                       # a teacher that likes nothing
    t[4, 1:] = -INF
    t[5] = 1e30
    loss, d = check_distill(z, index, t)
    assert loss[0] == INF and loss[1] == INF and loss[3] == 0 and (d[0] == 0).all() and (d[3] == 0).all()
    z[6, 11], t[7, 0] = float("nan"), float("nan")
    loss, stats = mfx.mfx_topk_distill_fwd(z, index, t)
    assert loss[6].isnan() and loss[7].isnan()


def test_distill_in_place_and_empty():
    for vocab, rows in ((5003, 40), (131072, 3), (131072, 200)):
        z = logits_of(rows, vocab, BF)
        index, t = lists_of(rows, vocab, 20, twice=True)
        w = torch.rand(rows, device=DEV)
        loss, want = mfx.mfx_topk_distill_fwd_bwd(z, index, t, w)
        loss2, stats = mfx.mfx_topk_distill_fwd(z, index, t)
        z2, want2 = z.clone(), mfx.mfx_topk_distill_bwd(w, z, index, t, stats)
        mfx.mfx_topk_distill_bwd(w, z2, index, t, stats, dlogits=z2)
        loss3, _ = mfx.mfx_topk_distill_fwd_bwd(z, index, t, w, dlogits=z)
        assert torch.equal(z, want) and torch.equal(z2, want2) and torch.equal(loss, loss3)
    z, w = logits_of(5, 77, F32), torch.rand(5, device=DEV)
    none = torch.empty((5, 0), device=DEV)
    loss, d = mfx.mfx_topk_distill_fwd_bwd(z, none.long(), none, w)
    assert (loss == 0).all() and (d == 0).all()
    z = torch.empty((5, 0), device=DEV)
    loss, d = mfx.mfx_topk_distill_fwd_bwd(z, torch.zeros((5, 2), dtype=torch.int64, device=DEV), torch.zeros((5, 2), device=DEV), w)
    assert (loss == 0).all() and d.shape == (5, 0)
    loss, d = mfx.mfx_topk_distill_fwd_bwd(torch.empty((0, 9), device=DEV), torch.zeros((0, 2), dtype=torch.int64, device=DEV), torch.zeros((0, 2), device=DEV), w[:0])
    assert loss.shape == (0,) and d.shape == (0, 9)


def test_gradients_against_differences():
    """Both losses' gradients against differences of the 64-bit forms."""
    z = logits_of(4, 500, F32)
    t = tokens_of(4, 500, lost=False)
    index, teacher = lists_of(4, 500, 9)
    g, ge = torch.randn(4, device=DEV), torch.randn(4, device=DEV)
    stats = mfx.mfx_token_logprobs_fwd(z, t, scale=0.9)[4]
    d1 = mfx.mfx_token_logprobs_bwd(g, ge, z, t, stats, scale=0.9).double()
    _, d2 = mfx.mfx_topk_distill_fwd_bwd(z, index, teacher, g, scale=0.9)

    def loss1(z):
        r, _, lp, _ = logprobs(z, t, 0.9)
        return (lp * g.double()).sum() + (r.entropy * ge.double()).sum()

    def loss2(z):
        return (distill(z, index, teacher, 0.9)[2] * g.double()).sum()

    v, s = torch.randn_like(z).double(), 1e-5
    for loss, d in ((loss1, d1), (loss2, d2.double())):
        by = (loss(z.double() + s * v) - loss(z.double() - s * v)) / (2 * s)
        # 32-bit gradients (a few 2^-22 of each term) and s^2 of third derivatives
        assert abs((d * v).sum() - by) <= 4e-6 * (d * v).abs().sum() + 1e-8


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("address", ["none", "off a vector"])
def test_rows_without_columns_lie_apart(dt, address):
    """Rows of no columns, a distance apart, in every number: nothing is read,
    and no entry or token counts."""
    L, k, ld = mfx.lib(), 3, 5
    some = torch.zeros(64, device=DEV)
    z = None if address == "none" else some.data_ptr() + 4
    for rows in (1, 7, 400):
        index = torch.zeros((rows, k), dtype=torch.int64, device=DEV)
        teacher, loss = torch.zeros((rows, k), device=DEV), torch.full((rows,), 7.0, device=DEV)
        lp, ent = torch.full((rows,), 7.0, device=DEV), torch.full((rows,), 7.0, device=DEV)
        s = torch.cuda.current_stream().cuda_stream
        assert L.mfx_topk_distill_fwd(dt, 0, rows, 0, ld, k, z, 64, index.data_ptr(), teacher.data_ptr(), None, 1.0,
                                      loss.data_ptr(), None, s) == 0
        assert (loss == 0).all()
        loss.fill_(7.0)
        assert L.mfx_topk_distill_fwd_bwd(dt, 0, rows, 0, ld, k, z, 64, index.data_ptr(), teacher.data_ptr(), None,
                                          teacher.data_ptr(), 1.0, loss.data_ptr(), None,
                                          ld, s) == 0
        assert (loss == 0).all()
        assert L.mfx_token_logprobs_fwd(dt, rows, 0, ld, z, 64, index.data_ptr(), 1.0, 0, lp.data_ptr(), ent.data_ptr(),
                                        None, None, None, None, None, s) == 0
        assert (lp == 0).all() and (ent == 0).all()
