"""The norm, the token log probabilities and the distillation as they are used:
one after another at a model's end against autograd in 64 bits, on other
streams than the current one, two at once, captured in graphs and replayed,
with workspaces of the caller's, and many rows of every kind."""
import math

import numpy as np
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import Rows, U, distill, distill_bwd, excess, half, logprobs, logprobs_bwd, top_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
INF = math.inf


def test_a_models_end():
    """h = x + residual; the norm; logits; a policy's loss and a distillation
    loss; and the gradients back to x, the residual and the weights."""
    torch.manual_seed(3)
    T, C, V, K = 48, 264, 1003, 12
    x, res = torch.randn(T, C, device=DEV), torch.randn(T, C, device=DEV)
    w, head = torch.rand(C, device=DEV) + 0.5, torch.randn(C, V, device=DEV) / C ** 0.5
    tokens = torch.randint(0, V, (T,), device=DEV)
    tokens[5] = -1
    index = torch.rand(T, V, device=DEV).topk(K, 1).indices
    teacher, g, ge, gd = torch.randn(T, K, device=DEV), torch.randn(T, device=DEV), torch.randn(T, device=DEV), torch.rand(T, device=DEV)

    y, h, rstd = mfx.mfx_add_rmsnorm_fwd(x, w, residual=res)
    logits = (y.double() @ head.double()).float()
    lp, ent, tv, ti, stats = mfx.mfx_token_logprobs_fwd(logits, tokens, scale=0.8, top=4)
    dz = mfx.mfx_token_logprobs_bwd(g, ge, logits, tokens, stats, scale=0.8).double()
    loss, d2 = mfx.mfx_topk_distill_fwd_bwd(logits, index, teacher, gd, scale=0.5)
    dz += d2.double()
    dy = (dz @ head.double().t()).float()
    dhead = y.double().t() @ dz
    dx, dres, dw = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, w, residual_dtype=F32)

    leaves = [t.double().requires_grad_() for t in (x, res, w, head)]
    x_, r_, w_, head_ = leaves
    hh = x_ + r_
    z = hh / torch.sqrt(hh.square().mean(1, keepdim=True) + 1e-6) * w_ @ head_
    logp = torch.log_softmax(z * 0.8, 1)
    keep = tokens >= 0
    plp = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    pent = -(logp.exp() * logp).sum(1)
    q = torch.softmax(teacher.double() * 0.5, 1)
    kl = (q * (q.log() - torch.log_softmax(z * 0.5, 1).gather(1, index))).sum(1)
    total = (torch.where(keep, plp * g + pent * ge, 0.0) + kl * gd).sum()
    want = torch.autograd.grad(total, leaves)
    # 32-bit norms and logits (2^-24 of each of some 300 terms) pass through the softmaxes' slopes of order one
    for a, b in ((lp, torch.where(keep, plp, 0.0)), (ent, torch.where(keep, pent, 0.0)), (loss, kl)):
        assert (a.double() - b).abs().max() <= 300 * U * (1 + b.abs().max())
    for a, b in zip((dx, dres, dw, dhead), want):
        assert (a.double() - b).norm() <= 300 * U * b.norm()
    assert torch.equal(ti.long()[keep], torch.topk(logits, 4, 1).indices[keep]) and (ti[5] == -1).all()


def calls(stream, rows):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, 520, generator=g).bfloat16().to(DEV)
    res, dh = torch.randn(rows, 520, generator=g).to(DEV), torch.randn(rows, 520, generator=g).to(DEV)
    w = torch.rand(520, generator=g).to(DEV)
    z = torch.randn(rows, 5003, generator=g).bfloat16().to(DEV)
    tokens = torch.randint(0, 5003, (rows,), generator=g).to(DEV)
    index, teacher = torch.randint(0, 5003, (rows, 9), generator=g).to(DEV), torch.randn(rows, 9, generator=g).to(DEV)
    gr = torch.randn(rows, generator=g).to(DEV)
    torch.cuda.synchronize()

    def run():
        kw = dict(stream=stream)
        y, h, rstd = mfx.mfx_add_rmsnorm_fwd(x, w, residual=res, **kw)
        q, scale, h2, r2 = mfx.mfx_add_rmsnorm_quant_fwd(x, w, residual=res, group=128, need_rstd=True, **kw)
        dx, dres, dw = mfx.mfx_add_rmsnorm_bwd(y, h, rstd, w, dh=dh, residual_dtype=F32, **kw)
        a = mfx.mfx_token_logprobs_fwd(z, tokens, top=7, **kw)
        d = mfx.mfx_token_logprobs_bwd(gr, gr, z, tokens, a[4], **kw)
        loss, st = mfx.mfx_topk_distill_fwd(z, index, teacher, **kw)
        d2 = mfx.mfx_topk_distill_bwd(gr, z, index, teacher, st, **kw)
        loss2, d3 = mfx.mfx_topk_distill_fwd_bwd(z, index, teacher, gr, **kw)
        return [y, h, rstd, q, scale, h2, r2, dx, dres, dw, *a, d, loss, st, d2, loss2, d3]

    return run


@pytest.mark.parametrize("rows", [40, 700])
@pytest.mark.parametrize("kind", ["stream", "handle", "default"])
def test_other_stream(kind, rows):
    want = calls(None, rows)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = {"stream": side, "handle": side.cuda_stream, "default": 0}[kind]
    run = calls(stream, rows)
    here = torch.cuda.current_stream() if kind != "default" else side
    other = side if kind != "default" else torch.cuda.default_stream()
    with torch.cuda.stream(here):
        with torch.cuda.stream(other):
            torch.cuda._sleep(20_000_000)  # about 10 ms: the calls wait in line
        got = run()
        for shift in range(9, 24):
            for _ in range(4):
                torch.empty(1 << shift, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_two_at_once():
    want = {n: calls(None, n)() for n in (40, 700)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    runs = [(n, calls(s, n)) for s, n in zip(streams, (700, 40, 700, 40))]
    got = [(n, run()) for _ in range(3) for n, run in runs]
    torch.cuda.synchronize()
    for n, outs in got:
        for i, (a, b) in enumerate(zip(outs, want[n])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (n, i)


@pytest.mark.parametrize("rows", [40, 700])
def test_graphs(rows):
    """Two captured graphs, replayed in turn and with eager calls between; new
    inputs in the same buffers."""
    eager = calls(None, rows)
    eager()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        run = calls(None, rows)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out, run))  # and what it reads
    want = eager()
    for _ in range(2):
        for graph, _, _ in graphs:
            graph.replay()
        eager()
    torch.cuda.synchronize()
    for _, out, _ in graphs:
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_given_outputs_and_workspaces():
    rows, V = 700, 5003
    z, tokens = torch.randn(rows, V, device=DEV), torch.randint(0, V, (rows,), device=DEV)
    want = mfx.mfx_token_logprobs_fwd(z, tokens, top=5)
    out = [torch.full_like(t, -7) for t in want]
    sizes = []

    def alloc(n):
        sizes.append(n)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)

    names = ("logprob", "entropy", "top_logprob", "top_index", "stats")
    got = mfx.mfx_token_logprobs_fwd(z, tokens, top=5, workspace=alloc, **dict(zip(names, out)))
    assert sizes[0] >= rows * 4 and all(a is b for a, b in zip(got, out))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    with pytest.raises(mfx.MfxError) as e:
        mfx.mfx_token_logprobs_fwd(z, tokens, top=5, workspace=none)
    assert e.value.status == 8
    few = mfx.mfx_token_logprobs_fwd(z[:9], tokens[:9], top=5, workspace=none)  # needs none
    assert torch.equal(few[3], want[3][:9])
    h, w = torch.randn(33, 512, device=DEV), torch.rand(512, device=DEV)
    rstd = torch.ones(33, device=DEV)
    a = mfx.mfx_add_rmsnorm_bwd(h, h, rstd, w, workspace=alloc)
    b = mfx.mfx_add_rmsnorm_bwd(h, h, rstd, w, dweight=torch.empty_like(w), dx=torch.empty_like(h))
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    with pytest.raises(mfx.MfxError):
        mfx.mfx_add_rmsnorm_bwd(h, h, rstd, w, workspace=none)


def test_refusals_of_the_binding():
    x, w = torch.randn(4, 64, device=DEV), torch.rand(64, device=DEV)
    z, t = torch.randn(4, 100, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    i, s = torch.zeros((4, 3), dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV)
    bad = [lambda: mfx.mfx_add_rmsnorm_fwd(x, w[:32]), lambda: mfx.mfx_add_rmsnorm_fwd(x.t(), w),
           lambda: mfx.mfx_add_rmsnorm_fwd(x, w, residual=x[:2]), lambda: mfx.mfx_add_rmsnorm_fwd(x, w, h=x),
           lambda: mfx.mfx_add_rmsnorm_fwd(x, w, y=x[:2]), lambda: mfx.mfx_add_rmsnorm_fwd(x, w, rstd=s[:2]),
           lambda: mfx.mfx_add_rmsnorm_fwd(w[0], w), lambda: mfx.mfx_add_rmsnorm_bwd(x, x, s, None, dweight=w),
           lambda: mfx.mfx_token_logprobs_fwd(z[0], t), lambda: mfx.mfx_token_logprobs_fwd(z.t(), t),
           lambda: mfx.mfx_token_logprobs_fwd(z, t[:2]), lambda: mfx.mfx_token_logprobs_fwd(z, t, top_index=i),
           lambda: mfx.mfx_token_logprobs_fwd(z[:1].expand(4, 100), t), lambda: mfx.mfx_topk_distill_fwd(z, i, z[:, :2].contiguous()),
           lambda: mfx.mfx_topk_distill_fwd(z, i, s), lambda: mfx.mfx_topk_distill_fwd_bwd(z, i, z[:, :3].contiguous(), s, dlogits=z[:2])]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mfx.mfx_add_rmsnorm_fwd(x.double(), w), lambda: mfx.mfx_add_rmsnorm_quant_fwd(x, w, q_dtype=BF),
                 lambda: mfx.mfx_token_logprobs_fwd(z, t.short()), lambda: mfx.mfx_token_logprobs_fwd(z, s),
                 lambda: mfx.mfx_add_rmsnorm_bwd(x, x, s, w, residual_dtype=BF),
                 lambda: mfx.mfx_topk_distill_fwd_bwd(z, i, z[:, :3].contiguous(), s, dlogits=z.to(BF))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: mfx.mfx_add_rmsnorm_fwd(x, w, eps=-1.0), lambda: mfx.mfx_add_rmsnorm_quant_fwd(x, w, group=64),
                 lambda: mfx.mfx_token_logprobs_fwd(z, t, top=65), lambda: mfx.mfx_token_logprobs_fwd(z, t, scale=0.0)):
        with pytest.raises(mfx.MfxError) as e:
            call()
        assert e.value.status == 9
    # numbers of other kinds count as the numbers that they are
    a = mfx.mfx_token_logprobs_fwd(z, t, scale=np.float64(0.5), top=np.int64(3))
    b = mfx.mfx_token_logprobs_fwd(z, t, scale=torch.tensor(0.5), top=3)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# --- many rows, which take kernels of their own ------------------------------
def many(rows, vocab, dtype, pad=0, lead=0):
    flat = (torch.randn(rows * (vocab + pad) + lead, device=DEV) * 3).to(dtype)
    z = flat[lead:].view(rows, vocab + pad)
    if pad:
        z[:, vocab:] = float("nan")
    return z[:, :vocab]


def check_many(z, tokens, scale, top):
    lp, ent, tv, ti, stats = mfx.mfx_token_logprobs_fwd(z, tokens, scale=scale, top=top)
    r, kept, want, tol = logprobs(z, tokens, scale)
    assert excess(lp, want, torch.where(kept, tol, 0.0)) <= 1
    assert excess(ent, torch.where(kept, r.entropy, 0.0), torch.where(kept, r.entropy_tol, 0.0)) <= 1
    if top:
        index = top_of(z, kept, top)
        assert torch.equal(ti.long(), index)
        value = torch.where(index < 0, -INF, r.logp.gather(1, index.clamp(min=0)))
        assert excess(tv, value, torch.where(index < 0, 0.0, r.logp_tol.gather(1, index.clamp(min=0)))) <= 1
    g, ge = torch.randn(z.shape[0], device=DEV), torch.randn(z.shape[0], device=DEV)
    d = mfx.mfx_token_logprobs_bwd(g, ge, z, tokens, stats, scale=scale)
    want, tol = logprobs_bwd(r, kept, tokens, g, ge, scale)
    assert excess(d, want, tol + want.abs() * half(z.dtype)) <= 1


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,lead", [(0, 0), (3, 1), (13, 7), (8, 5)])
@pytest.mark.parametrize("vocab", [1, 5, 8, 17, 130, 1000, 4099, 8192, 20011])
def test_many_rows(vocab, pad, lead, dtype):
    rows = 1300 if vocab < 5000 else 640
    z = many(rows, vocab, dtype, pad, lead)
    tokens = torch.randint(-1, vocab + 1, (rows,), device=DEV)  # some rows left out, next to each other too
    tokens[100:600] = -1
    check_many(z, tokens, 0.9, 5)
    index = torch.randint(-1, vocab + 1, (rows, 7), device=DEV)
    t = torch.randn((rows, 7), device=DEV).to(dtype)
    r, q, want, tol, q_tol = distill(z, index, t, 1.1)
    loss, stats = mfx.mfx_topk_distill_fwd(z, index, t, scale=1.1)
    assert excess(loss, want, tol) <= 1
    g = torch.randn(rows, device=DEV)
    d = mfx.mfx_topk_distill_bwd(g, z, index, t, stats, scale=1.1)
    d_want, d_tol = distill_bwd(r, q, q_tol, index, g, 1.1, vocab)
    assert excess(d, d_want, d_tol + d_want.abs() * half(dtype)) <= 1


@pytest.mark.parametrize("vocab,dtype,top", [(300007, BF, 20), (300007, BF, 64), (160001, F32, 30)])
def test_many_long_rows(vocab, dtype, top):
    z = many(307, vocab, dtype, 1)
    tokens = torch.randint(0, vocab, (307,), device=DEV)
    check_many(z, tokens, 1.0, top)


@pytest.mark.parametrize("vocab", [300, 5000, 66000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_masked_rows(vocab, dtype):
    z = many(8, vocab, dtype)
    z[0] = -INF
    z[1] = -INF
    z[1, vocab // 3] = 2.0
    z[2, ::2] = -INF
    z[3] = torch.finfo(dtype).min
    z[4, 5:] = torch.finfo(dtype).min
    z[5] = 0.0
    z[6] = torch.finfo(dtype).max / 4
    z[7, :] = -INF
    z[7, -3:] = torch.tensor([1.0, -0.0, 0.0], dtype=dtype)
    t = torch.tensor([0, vocab // 3, 1, 2, 0, 9, 3, vocab - 1], device=DEV)
    z, t = z.repeat(60, 1), t.repeat(60)
    for scale, top in ((0.5, 10), (3.0, 64), (1.0, 0)):
        check_many(z, t, scale, top)
    z[0, 17], z[1, 100], z[2, 3] = float("nan"), INF, float("nan")
    t[2] = -1
    lp, ent, tv, ti, stats = mfx.mfx_token_logprobs_fwd(z, t, top=4)
    assert lp[:2].isnan().all() and ent[:2].isnan().all() and lp[2] == 0 and ti[1, 0] == 100 and (ti[2] == -1).all()
    assert 17 not in ti[0].tolist()


def test_many_rows_of_ties_and_orders():
    for vocab in (900, 40000, 131072):
        rise = torch.arange(vocab, device=DEV, dtype=F32)
        place = torch.arange(vocab, device=DEV)
        z = torch.stack([rise, -rise, torch.where(place % 1024 < 8, 100.0, 0.0) + torch.rand(vocab, device=DEV),
                         torch.where(place % 512 < 16, rise, -rise), torch.randint(0, 3, (vocab,), device=DEV).float(),
                         torch.where(place % 4096 == 0, 1.0, -INF), torch.zeros(vocab, device=DEV),
                         (place % 7).float()]).repeat(50, 1)
        for rows in (z, z.to(BF)):
            for top in (1, 24, 25, 64):
                t = torch.zeros(rows.shape[0], dtype=torch.int64, device=DEV)
                ti = mfx.mfx_token_logprobs_fwd(rows, t, top=top, need_stats=False)[3]
                assert torch.equal(ti.long(), top_of(rows, t >= 0, top))


def test_offsets_past_32_bits():
    """Rows whose first element lies past 2^31 elements from the buffer's."""
    rows, vocab = 66000, 33000  # 2.18e9 bf16 logits
    z = torch.empty((rows, vocab), dtype=BF, device=DEV)
    z[:].normal_()
    tokens = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
    some = torch.tensor([0, 1, 32999, 65534, 65999], device=DEV)
    tokens[some] = torch.tensor([5, 32999, 7, 0, 100], device=DEV)
    lp, ent, tv, ti, stats = mfx.mfx_token_logprobs_fwd(z, tokens, top=3)
    small, ts = z[some].contiguous(), tokens[some]
    r, kept, want, tol = logprobs(small, ts, 1.0)
    assert excess(lp[some], want, tol) <= 1 and torch.equal(ti[some].long(), top_of(small, kept, 3))
    assert (lp != 0).sum() == 5
    g = torch.ones(rows, device=DEV)
    d = mfx.mfx_token_logprobs_bwd(g, None, z, tokens, stats, dlogits=z)  # in place
    want, tol = logprobs_bwd(r, kept, ts, g[some], None, 1.0)
    assert excess(d[some], want, tol + want.abs() * half(BF)) <= 1
    tokens[some] = 0
    assert not d[1000].any() and not d[65998].any()
    del d, z
    x = torch.empty((rows, vocab), dtype=BF, device=DEV)
    x[:].normal_()
    y, _, rstd = mfx.mfx_add_rmsnorm_fwd(x, None)
    want = x[some].double() / torch.sqrt(x[some].double().square().mean(1, keepdim=True) + 1e-6)
    assert excess(y[some], want, want.abs() * (half(BF) + 64 * U)) <= 1
