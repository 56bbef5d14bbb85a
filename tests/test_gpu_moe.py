"""Tokens sorted by expert and back, with weights applied, and the gradients.

The maps and the copies are exact.  Sums over a token's rows are fp32
fused multiply-adds in choice order: at most topk roundings of the sum of
magnitudes, then one to the output dtype.  dweight is one fp32 dot product of
cols products, at most cols / 256 + 8 of them in a row to a thread and 12 joins:
bounded by (cols / 256 + 24) half steps of the sum of magnitudes."""
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def choices(tokens, topk, experts, seed=0, lost=0.1):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, experts, (tokens, topk), generator=g)
    bad = torch.rand((tokens, topk), generator=g)
    e[bad < lost / 2] = -1
    e[(bad >= lost / 2) & (bad < lost)] = experts + 3  # also no expert
    return e.to(torch.int32)


def plain_sort(expert_of, experts, align, capacity, rows):
    tokens, topk = expert_of.shape
    lists = [[] for _ in range(experts)]
    for s, e in enumerate(expert_of.view(-1).tolist()):
        if 0 <= e < experts and (not capacity or len(lists[e]) < capacity):
            lists[e].append(s)
    row_of, slot_of, offsets = [-1] * (tokens * topk), [-1] * rows, [0]
    for mine in lists:
        for i, s in enumerate(mine):
            row_of[s] = offsets[-1] + i
            slot_of[offsets[-1] + i] = s
        offsets.append(offsets[-1] + -(-len(mine) // align) * align)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)
    return i32(row_of).view(tokens, topk), i32(slot_of), i32(offsets), i32([len(m) for m in lists])


def sort(e, experts, **kw):
    return mfx.mfx_moe_sort(e.to(DEV), experts, **kw)


@pytest.mark.parametrize("align", [1, 16, 128])
@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 64), (7, 2, 3), (64, 8, 256), (300, 6, 60),
                                                 (1025, 2, 8), (5000, 8, 128), (3000, 1, 4096), (40000, 8, 17)])
def test_sort(tokens, topk, experts, align):
    e = choices(tokens, topk, experts, seed=tokens)
    for capacity in (0, 1, max(1, tokens * topk // experts)):
        got = sort(e, experts, align=align, capacity=capacity)
        want = plain_sort(e, experts, align, capacity, mfx.mfx_moe_rows(tokens, topk, experts, align))
        for a, b, name in zip(got, want, ("row_of", "slot_of", "offsets", "counts")):
            assert torch.equal(a.cpu(), b), (name, capacity)


def test_sort_one_expert_and_none():
    e = torch.zeros(9000, 3, dtype=torch.int32)
    for value in (0, 5, -1):
        e.fill_(value)
        got = sort(e, 6, align=8)
        want = plain_sort(e, 6, 8, 0, mfx.mfx_moe_rows(9000, 3, 6, 8))
        for a, b in zip(got, want):
            assert torch.equal(a.cpu(), b)


def test_sort_without_tokens():
    for shape in ((0, 4), (5, 0)):
        row_of, slot_of, offsets, counts = sort(torch.empty(shape, dtype=torch.int32), 3, rows=10)
        assert row_of.shape == shape and (slot_of == -1).all() and not offsets.any() and not counts.any()


def test_sort_with_capacity_rows():
    """With a capacity the sorted buffers may be as small as it allows."""
    e = choices(500, 4, 5, seed=3)
    got = sort(e, 5, align=8, capacity=30, rows=160)
    want = plain_sort(e, 5, 8, 30, 160)
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)
    with pytest.raises(mfx.MfxError):
        sort(e, 5, align=8, capacity=30, rows=159)


def off(t, k):
    buf = torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)
    v = buf[k:].view(t.shape)
    v.copy_(t)
    return v


SHAPES = [(1, 1, 1, 8), (3, 2, 4, 1), (5, 2, 3, 7), (16, 8, 64, 4096), (130, 2, 8, 1024), (77, 9, 12, 333),
          (200, 4, 16, 2056), (60, 6, 60, 4099), (33, 17, 40, 72)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("align", [1, 16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_there_and_back(shape, align, dtype, shift):
    tokens, topk, experts, cols = shape
    e = choices(tokens, topk, experts, seed=cols)
    capacity = max(1, tokens * topk * 3 // (experts * 2))
    row_of, slot_of, _, _ = sort(e, experts, align=align, capacity=capacity)
    rows = slot_of.numel()
    g = torch.Generator().manual_seed(cols + 1)
    new = lambda *s: torch.randn(s, generator=g)
    put = lambda t, d=dtype: off(t.to(d).to(DEV), shift)
    x, gy, y, gr = put(new(tokens, cols)), put(new(tokens, cols)), put(new(rows, cols)), put(new(rows, cols))
    w, gw = put(new(tokens, topk), F32), put(new(rows), F32)
    has = (row_of >= 0)
    r = row_of.clamp(min=0).long()
    pad = slot_of < 0
    half = torch.finfo(dtype).eps / 2

    out, ow = mfx.mfx_moe_permute_fwd(x, row_of, slot_of, weight=w)
    tok = slot_of.clamp(min=0).long() // topk
    assert torch.equal(out, x[tok].masked_fill(pad[:, None], 0)) and torch.equal(
        ow, w.view(-1)[slot_of.clamp(min=0).long()].masked_fill(pad, 0))
    bare, none = mfx.mfx_moe_permute_fwd(x, row_of, slot_of)
    assert none is None and torch.equal(bare, out)

    dx, dw = mfx.mfx_moe_permute_bwd(gr, row_of, g_weight=gw)
    parts = gr.double()[r].masked_fill(~has[..., None], 0)
    want, size = parts.sum(1), parts.abs().sum(1)
    assert ((dx.double() - want).abs() <= half * want.abs() + (topk * U * (1 + half)) * size).all()
    assert torch.equal(dw, gw[r].masked_fill(~has, 0))

    for weight in (w, None):
        z = mfx.mfx_moe_unpermute_fwd(y, row_of, weight=weight)
        f = weight.double()[..., None] if weight is not None else 1.0
        parts = y.double()[r].masked_fill(~has[..., None], 0) * f
        want, size = parts.sum(1), parts.abs().sum(1)
        assert ((z.double() - want).abs() <= half * want.abs() + (topk * U * (1 + half)) * size).all()

        dy, dw = mfx.mfx_moe_unpermute_bwd(gy, y, row_of, slot_of, weight=weight)
        f = w.view(-1)[slot_of.clamp(min=0).long()][:, None] if weight is not None else 1.0
        want = (gy.float()[tok] * f).to(dtype).masked_fill(pad[:, None], 0)
        assert torch.equal(dy, want)
        if weight is None:
            assert dw is None
            continue
        prod = gy.double()[:, None] * y.double()[r]
        want = prod.sum(-1).masked_fill(~has, 0)
        tol = (cols / 256 + 24) * U * prod.abs().sum(-1)
        assert ((dw.double() - want).abs() <= tol).all() and not dw[~has].any()
        alone, _ = mfx.mfx_moe_unpermute_bwd(gy, None, row_of, slot_of, weight=weight, need_dweight=False)
        assert torch.equal(alone, dy)


def test_padding_does_not_leak():
    """NaN in padding rows of y and g stays there."""
    e = choices(50, 2, 4, seed=5)
    row_of, slot_of, _, _ = sort(e, 4, align=16)
    y = torch.randn(slot_of.numel(), 256, device=DEV)
    y[slot_of < 0] = float("nan")
    w, g = torch.rand(50, 2, device=DEV), torch.randn(50, 256, device=DEV)
    dy, dw = mfx.mfx_moe_unpermute_bwd(g, y, row_of, slot_of, weight=w)
    for t in (mfx.mfx_moe_unpermute_fwd(y, row_of, weight=w), mfx.mfx_moe_permute_bwd(y, row_of)[0], dy, dw):
        assert torch.isfinite(t).all()


def test_maps_out_of_range_count_as_none():
    row_of = torch.tensor([[0, 7], [-5, 2]], dtype=torch.int32, device=DEV)
    slot_of = torch.tensor([0, 99, 3], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 16, device=DEV)
    out, _ = mfx.mfx_moe_permute_fwd(x, row_of, slot_of)
    assert torch.equal(out[0], x[0]) and not out[1].any() and torch.equal(out[2], x[1])
    y = torch.randn(3, 16, device=DEV)
    z = mfx.mfx_moe_unpermute_fwd(y, row_of)
    assert torch.equal(z[0], y[0]) and torch.equal(z[1], y[2])


def test_same_bits_again_and_on_another_stream():
    e = choices(3000, 4, 16, seed=9)
    x, y = torch.randn(3000, 1000, device=DEV), torch.randn(12000, 1000, device=DEV)
    w = torch.rand(3000, 4, device=DEV)

    def step():
        row_of, slot_of, o, c = sort(e, 16)
        xp, wp = mfx.mfx_moe_permute_fwd(x, row_of, slot_of, weight=w)
        return [row_of, slot_of, o, c, xp, wp, mfx.mfx_moe_unpermute_fwd(y, row_of, weight=w),
                *mfx.mfx_moe_unpermute_bwd(x, y, row_of, slot_of, weight=w)]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_graph_capture():
    """Sort, permute and back in one graph, replayed on new choices."""
    e1, e2 = choices(900, 4, 16, seed=10).to(DEV), choices(900, 4, 16, seed=11).to(DEV)
    x, w = torch.randn(900, 512, device=DEV, dtype=BF), torch.rand(900, 4, device=DEV)
    e = e1.clone()
    rows = mfx.mfx_moe_rows(900, 4, 16, 8)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)
    maps = dict(row_of=i32(900, 4), slot_of=i32(rows), offsets=i32(17), counts=i32(16))
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    xp, wp = torch.empty(rows, 512, device=DEV, dtype=BF), torch.empty(rows, device=DEV)
    z = torch.empty_like(x)

    def step():
        mfx.mfx_moe_sort(e, 16, align=8, workspace=ws, **maps)
        mfx.mfx_moe_permute_fwd(x, maps["row_of"], maps["slot_of"], weight=w, out=xp, out_weight=wp)
        mfx.mfx_moe_unpermute_fwd(xp, maps["row_of"], weight=w, out=z)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for src in (e2, e1):
        e.copy_(src)
        graph.replay()
        got = [t.clone() for t in (*maps.values(), xp, wp, z)]
        step()
        for a, b in zip(got, (*maps.values(), xp, wp, z)):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """Forward and backward of the weighted way back are each other's transposes."""
    e = choices(20, 3, 5, seed=12)
    row_of, slot_of, _, _ = sort(e, 5, align=4)
    g = torch.Generator().manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g).to(DEV)
    y, w, up = new(slot_of.numel(), 40), new(20, 3), new(20, 40)
    dy, dw = mfx.mfx_moe_unpermute_bwd(up, y, row_of, slot_of, weight=w)
    loss = lambda y, w: (mfx.mfx_moe_unpermute_fwd(y, row_of, weight=w).double() * up.double()).sum().item()
    h = 0.25  # the sum is linear in y and in w
    for at in [(0, 0), (1, 39), (7, 5)]:
        d = torch.zeros_like(y)
        d[at] = h
        assert abs((loss(y + d, w) - loss(y - d, w)) / (2 * h) - dy[at].item()) <= 1e-4
    for at in [(0, 0), (3, 2), (19, 1)]:
        d = torch.zeros_like(w)
        d[at] = h
        assert abs((loss(y, w + d) - loss(y, w - d)) / (2 * h) - dw[at].item()) <= 1e-4


def test_empty():
    row_of, slot_of = torch.empty((0, 2), dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 16, device=DEV)
    assert mfx.mfx_moe_permute_fwd(x, row_of, slot_of)[0].shape == (0, 16)
    assert mfx.mfx_moe_unpermute_fwd(x, row_of).shape == (0, 16)
    # tokens without rows
    row_of = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    assert not mfx.mfx_moe_unpermute_fwd(x, row_of).any()
    dy, dw = mfx.mfx_moe_unpermute_bwd(torch.randn(3, 16, device=DEV), x, row_of, slot_of,
                                       weight=torch.rand(3, 2, device=DEV))
    assert dy.shape == (0, 16) and not dw.any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_zero_width(dtype):
    """Rows without columns still carry their weights, and a product of no
    columns is zero: every fp32 output is written (they hold NaN before)."""
    e = choices(37, 3, 5, seed=13)
    row_of, slot_of, _, _ = sort(e, 5, align=8)
    rows = slot_of.numel()
    x, y = torch.empty(37, 0, device=DEV, dtype=dtype), torch.empty(rows, 0, device=DEV, dtype=dtype)
    w, gw = torch.rand(37, 3, device=DEV), torch.rand(rows, device=DEV)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)
    has, pad = row_of >= 0, slot_of < 0
    out, ow = mfx.mfx_moe_permute_fwd(x, row_of, slot_of, weight=w, out_weight=nan(rows))
    assert out.shape == (rows, 0)
    assert torch.equal(ow, w.view(-1)[slot_of.clamp(min=0).long()].masked_fill(pad, 0))
    dx, dw = mfx.mfx_moe_permute_bwd(y, row_of, g_weight=gw, dweight=nan(37, 3))
    assert dx.shape == (37, 0) and torch.equal(dw, gw[row_of.clamp(min=0).long()].masked_fill(~has, 0))
    for weight in (w, None):
        dy, dw = mfx.mfx_moe_unpermute_bwd(x, y, row_of, slot_of, weight=weight, dweight=nan(37, 3))
        assert dy.shape == (rows, 0) and torch.equal(dw, torch.zeros_like(w))
    assert mfx.mfx_moe_unpermute_fwd(y, row_of, weight=w).shape == (37, 0)
