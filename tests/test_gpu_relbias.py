"""Softmax of attention scores with a learned relative position bias and
dropout, forward and backward, against the plain 64-bit form."""
import math

import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from relbias_ref import close, reference

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def offset_view(t, k):
    """A contiguous tensor equal to t that begins k elements into its buffer."""
    buf = torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)
    v = buf[k:].view(t.shape)
    v.copy_(t)
    return v


def inputs(b, np_, sq, sk, dtype, seed=0, buckets=32, table_dtype=None, mask=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((b, np_, sq, sk), generator=g) * 8).to(dtype).to(DEV)
    dy = torch.randn((b, np_, sq, sk), generator=g).to(dtype).to(DEV)
    table = torch.randn((buckets, np_), generator=g).to(table_dtype or dtype).to(DEV) if buckets else None
    m = None
    if mask == "pad":
        n = torch.randint(1, sk + 1, (b,), generator=g)
        m = torch.where(torch.arange(sk) < n[:, None], 0.0, -math.inf).reshape(b, 1, 1, sk).to(dtype).to(DEV)
    elif mask == "full":
        m = torch.randn((b, np_, sq, sk), generator=g)
        m[torch.rand(m.shape, generator=g) < 0.2] = -math.inf
        m = m.to(dtype).to(DEV)
    elif mask == "heads":
        m = torch.randn((1, np_, 1, sk), generator=g).to(dtype).to(DEV)
    return x, dy, table, m


def run_both(x, dy, scale=0.125, **kw):
    y, stats = mfx.mfx_relbias_softmax_dropout_fwd(x, scale, **kw)
    dx, dt = mfx.mfx_relbias_softmax_dropout_bwd(dy, x, stats, scale, **kw)
    return y, stats, dx, dt


def check(x, dy, scale=0.125, **kw):
    y, stats, dx, dt = run_both(x, dy, scale, **kw)
    ry, ty, rdx, tdx, rdt, tdt = reference(x, scale, dy=dy, **kw)
    close(y, ry, ty, "y")
    close(dx, rdx, tdx, "dx")
    if rdt is not None:
        close(dt, rdt, tdt, "dtable")
    bare, none = mfx.mfx_relbias_softmax_dropout_fwd(x, scale, need_stats=False, **kw)
    assert none is None and torch.equal(bare.view(torch.uint8), y.view(torch.uint8))
    return y, dx, dt


SIZES = [(1, 1, 1, 1), (2, 3, 1, 2), (1, 2, 3, 5), (2, 1, 7, 8), (1, 3, 33, 31), (2, 2, 64, 64), (1, 2, 5, 257),
         (3, 2, 20, 300), (1, 5, 17, 1000), (2, 1, 9, 1025), (1, 2, 40, 2048), (1, 1, 3, 4099), (1, 1, 2, 8200),
         (1, 2, 2, 20001)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(size, dtype):
    x, dy, table, _ = inputs(*size, dtype, seed=sum(size))
    check(x, dy, table=table, q_start=max(0, size[3] - size[2]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [(1, 1, 1, 1), (2, 3, 33, 31), (2, 2, 20, 300), (1, 2, 9, 2056), (1, 1, 2, 9001)])
@pytest.mark.parametrize("p,base", [(0.1, 0), (0.5, 8 * (1 << 33)), (0.25, 12345678901)])
def test_dropout(size, dtype, p, base):
    x, dy, table, m = inputs(*size, dtype, seed=3, mask="pad")
    check(x, dy, table=table, mask=m, p=p, seed=987654321012, offset=77, elem_base=base)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask", ["pad", "full", "heads"])
@pytest.mark.parametrize("sq,sk", [(4, 6), (19, 129), (6, 1300)])
def test_masks(mask, sq, sk, dtype):
    x, dy, table, m = inputs(3, 2, sq, sk, dtype, seed=4, mask=mask)
    check(x, dy, table=table, mask=m, q_start=2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("sq,sk,start", [(64, 64, 0), (40, 300, 260), (40, 300, -10), (5, 1200, 4000), (300, 40, -200)])
def test_causal(sq, sk, start, two, dtype):
    """Queries before the first key (empty rows), inside, and past the last."""
    x, dy, table, m = inputs(2, 2, sq, sk, dtype, seed=5, mask="pad")
    nan = torch.arange(sk, device=DEV) > start + torch.arange(sq, device=DEV)[:, None]
    x.masked_fill_(nan, math.nan)  # what is left out is not read
    dy.masked_fill_(nan, math.nan)
    kw = dict(table=table, mask=m, causal=True, bidirectional=two, q_start=start, p=0.1, seed=5)
    y, dx, _ = run_both(x, dy, **kw)[0:4:2] + (None,)
    clean = torch.nan_to_num(x, nan=0.0), torch.nan_to_num(dy, nan=0.0)
    ry, ty, rdx, tdx, rdt, tdt = reference(clean[0], 0.125, dy=clean[1], **kw)
    close(y, ry, ty, "y")
    close(dx, rdx, tdx, "dx")
    assert not y[..., nan].any() and not dx[..., nan].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequence_starts(dtype):
    """Each sequence at its own position, one before all keys, one after."""
    x, dy, table, _ = inputs(4, 3, 2, 700, dtype, seed=6)
    at = torch.tensor([0, 333, -5, 2000], dtype=torch.int32, device=DEV)
    y, _, _ = check(x, dy, table=table, causal=True, bidirectional=False, seq_start=at, q_start=1)
    assert not y[2].any()  # positions -4 and -3: nothing to look at


@pytest.mark.parametrize("buckets,far,two", [(2, 2, False), (4, 2, True), (5, 17, False), (32, 128, True),
                                             (32, 128, False), (64, 800, True), (256, 2048, True), (128, 2048, False),
                                             (6, 9, True), (16, 9, False)])
def test_bucket_functions(buckets, far, two):
    """Every border of the bucket function, by a one-hot row's bias and its gradient."""
    x, dy, table, _ = inputs(1, 2, 3, 1500, F32, seed=7, buckets=buckets)
    check(x, dy, table=table, max_distance=far, bidirectional=two, q_start=750)
    if far > 1000:
        x, dy, table, _ = inputs(1, 1, 2, 5000, F32, seed=8, buckets=buckets)
        check(x, dy, table=table, max_distance=far, bidirectional=two, q_start=2400)


def test_bucket_borders_exact():
    """One finite score per row at each distance: y is one there, and the
    gradient of the table tells its bucket."""
    sk, num = 400, 32
    for two in (True, False):
        x = torch.zeros(1, 1, 1, sk, device=DEV)
        table = torch.arange(num, dtype=F32, device=DEV).view(num, 1) / 8
        y, _ = mfx.mfx_relbias_softmax_dropout_fwd(x, 1.0, table=table, bidirectional=two, q_start=200)
        got = (torch.log(y.double().view(-1)) * 8)
        from relbias_ref import bucket
        want = bucket(torch.arange(sk, device=DEV) - 200, num, 128, two)
        assert torch.equal((got - got[200]).round().long(), want - want[200])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_table(dtype):
    x, dy, _, m = inputs(2, 2, 9, 333, dtype, seed=9, buckets=0, mask="pad")
    _, _, dt = check(x, dy, mask=m, p=0.1, seed=3)
    assert dt is None


@pytest.mark.parametrize("dtype,table_dtype", [(BF, F32), (F32, BF)])
def test_table_dtypes(dtype, table_dtype):
    x, dy, table, _ = inputs(2, 2, 9, 333, dtype, seed=10, table_dtype=table_dtype)
    _, _, dt = check(x, dy, table=table)
    assert dt.dtype == table_dtype


@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_rows_and_hidden_values(dtype):
    """Rows whose mask leaves nothing are zeros; NaN and infinities under a
    mask of -inf, and in the gradient there, have no effect."""
    x, dy, table, _ = inputs(2, 2, 5, 300, dtype, seed=11)
    m = torch.zeros(2, 1, 5, 300, device=DEV, dtype=dtype)
    m[0, :, 2] = -math.inf
    m[..., 100:140] = -math.inf
    y0, dx0, dt0 = check(x, dy, table=table, mask=m, p=0.1, seed=1)
    assert not y0[0, :, 2].any() and not dx0[0, :, 2].any()
    x[..., 100:120], x[..., 120:140] = math.nan, math.inf
    dy[..., 100:110], dy[..., 110:140] = math.nan, -math.inf
    y, _, dx, dt = run_both(x, dy, table=table, mask=m, p=0.1, seed=1)
    assert torch.equal(y, y0) and torch.equal(dx, dx0) and torch.equal(dt, dt0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sk", [40, 300, 5000])
def test_lowest_masks(sk, dtype):
    """Padding by the type's lowest value; rows that see nothing else are the
    softmax of their scores, as the addition says."""
    x, dy, table, _ = inputs(2, 2, 6, sk, dtype, seed=12)
    m = torch.zeros(2, 1, 6, sk, device=DEV, dtype=dtype)
    m[..., sk // 2:] = torch.finfo(dtype).min
    m[:, :, 1] = torch.finfo(dtype).min
    m[:, :, 2] = -1e5
    check(x, dy, table=table, mask=m)
    check(x, dy, table=table, mask=m, causal=True, bidirectional=False, q_start=sk // 4, p=0.1, seed=2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_and_infinite_scores(dtype):
    """A NaN or +inf score makes its row NaN, -inf excludes its key."""
    x, dy, table, _ = inputs(1, 1, 4, 900, dtype, seed=13)
    x[0, 0, 0, 5], x[0, 0, 1, 700], x[0, 0, 2, 30:60] = math.nan, math.inf, -math.inf
    y, _, dx, _ = run_both(x, dy, table=table)
    ry, ty, rdx, tdx, _, _ = reference(x, 0.125, table=table, dy=dy)
    assert torch.isnan(y[0, 0, :2]).all() and torch.isnan(dx[0, 0, :2]).all()
    close(y[:, :, 2:], ry[:, :, 2:], ty[:, :, 2:], "y")
    close(dx[:, :, 2:], rdx[:, :, 2:], tdx[:, :, 2:], "dx")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b,np_,sk", [(1, 8, 77), (3, 4, 2000), (2, 2, 9000), (1, 3, 40000), (1, 2, 131081)])
def test_single_tokens(b, np_, sk, dtype):
    x, _, table, m = inputs(b, np_, 1, sk, dtype, seed=14, mask="pad")
    kw = dict(table=table, bidirectional=False, q_start=sk - 1)
    for more in ({}, {"mask": m}, {"causal": True, "seq_start": torch.tensor([-3 * i for i in range(b)],
                                                                          dtype=torch.int32, device=DEV)}):
        y, none = mfx.mfx_relbias_softmax_dropout_fwd(x, 0.125, need_stats=False, **kw, **more)
        ry, ty = reference(x, 0.125, **kw, **more)
        close(y, ry, ty, "y")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_any_alignment(off, dtype):
    x, dy, table, m = inputs(2, 2, 7, 264, dtype, seed=15, mask="full")
    kw = dict(table=table, mask=m, p=0.1, seed=4)
    want = run_both(x, dy, **kw)
    kw["mask"], kw["table"] = offset_view(m, off), offset_view(table, 1)
    got = run_both(offset_view(x, off), offset_view(dy, 2 * off), **kw)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    close(got[3], want[3].double(), 1e-2 * want[3].double().abs() + 1e-3, "dtable")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sk", [200, 9000])
def test_in_place(sk, dtype):
    x, dy, table, _ = inputs(2, 2, 5, sk, dtype, seed=16)
    kw = dict(table=table, p=0.1, seed=4)
    y, stats, dx, dt = run_both(x, dy, **kw)
    z = x.clone()
    mfx.mfx_relbias_softmax_dropout_fwd(z, 0.125, y=z, need_stats=False, **kw)
    assert torch.equal(z, y)
    for which in ("dy", "x"):
        a, b = x.clone(), dy.clone()
        out, dt2 = mfx.mfx_relbias_softmax_dropout_bwd(b, a, stats, 0.125, dx=b if which == "dy" else a, **kw)
        assert torch.equal(out, dx) and torch.equal(dt2, dt)


def test_same_bits_again_and_on_another_stream():
    x, dy, table, m = inputs(2, 4, 300, 515, BF, seed=17, mask="pad")
    kw = dict(table=table, mask=m, p=0.1, seed=4)
    first = run_both(x, dy, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run_both(x, dy, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_shards_share_one_mask():
    """Batches processed apart with their own elem_base drop the same elements."""
    x, dy, table, _ = inputs(3, 2, 11, 123, BF, seed=18)
    whole, _ = mfx.mfx_relbias_softmax_dropout_fwd(x, 0.125, table=table, p=0.3, seed=9)
    for i in range(3):
        part, _ = mfx.mfx_relbias_softmax_dropout_fwd(x[i:i + 1], 0.125, table=table, p=0.3, seed=9,
                                                      elem_base=i * 2 * 11 * 123)
        assert torch.equal(part[0], whole[i])


def test_empty():
    table = torch.randn(32, 2, device=DEV)
    for shape in ((0, 2, 3, 5), (2, 2, 0, 5), (2, 2, 3, 0)):
        x = torch.empty(shape, device=DEV)
        y, stats, dx, dt = run_both(x, x.clone(), table=table)
        assert y.shape == shape and dx.shape == shape and not dt.any()


def test_gradient_against_differences():
    """d(sum w y) by central differences of the 64-bit form at a few places."""
    x, w, table, _ = inputs(1, 2, 4, 40, F32, seed=19)
    kw = dict(table=table, p=0.25, seed=6, q_start=20)
    _, _, dx, dt = run_both(x, w, **kw)
    h = 1e-5
    loss = lambda x, t: (reference(x, 0.125, **{**kw, "table": t})[0] * w.double()).sum().item()
    for at in [(0, 0, 0, 0), (0, 1, 2, 21), (0, 1, 3, 39)]:
        e = torch.zeros_like(x, dtype=torch.float64)
        e[at] = h
        num = (loss(x.double() + e, table) - loss(x.double() - e, table)) / (2 * h)
        assert abs(num - dx[at].item()) <= 1e-6
    for at in [(0, 0), (3, 1), (20, 0)]:
        e = torch.zeros_like(table, dtype=torch.float64)
        e[at] = h
        num = (loss(x.double(), table.double() + e) - loss(x.double(), table.double() - e)) / (2 * h)
        assert abs(num - dt[at].item()) <= 1e-5


def test_graph_capture():
    x, dy, table, m = inputs(2, 2, 40, 300, BF, seed=20, mask="pad")
    kw = dict(table=table, mask=m, p=0.1, seed=4)
    want = run_both(x, dy, **kw)
    y, stats, dx, dt = (torch.empty_like(t) for t in want)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def step():
        mfx.mfx_relbias_softmax_dropout_fwd(x, 0.125, y=y, stats=stats, **kw)
        mfx.mfx_relbias_softmax_dropout_bwd(dy, x, stats, 0.125, dx=dx, dtable=dt, workspace=ws, **kw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (y, stats, dx, dt):
        t.zero_()
    g.replay()
    for a, b in zip((y, stats, dx, dt), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("scale", [0.125, 0.0884, -0.3, 0.0])
def test_one_key_has_no_gradient(scale, p, dtype):
    """Where one key takes part (by length, position or mask) P is exactly one
    and the gradient exactly zero, as the difference says."""
    for sk, mask, causal in ((1, None, False), (9, "one", False), (300, "one", False), (40, None, True)):
        x, dy, table, _ = inputs(2, 3, 1 if causal else 6, sk, dtype, seed=sk)
        m = None
        if mask:
            m = torch.full((2, 1, 6, sk), -math.inf, device=DEV, dtype=dtype)
            m[..., sk // 2] = 0
            m[:, :, 3] = torch.finfo(dtype).min  # next to the lowest value, -inf
            m[:, :, 3, :sk // 2] = m[:, :, 3, sk // 2 + 1:] = -math.inf
        y, _, dx, dt = run_both(x, dy, scale, table=table, mask=m, causal=causal, bidirectional=not causal, p=p, seed=7)
        if p == 0:
            assert ((y == 0) | (y == 1)).all()
        assert not dx.any() and not dt.any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-35, 1.0])
def test_scales(scale, dtype):
    x, dy, table, m = inputs(2, 2, 7, 130, dtype, seed=21, mask="pad")
    check(x, dy, scale, table=table, mask=m, p=0.1, seed=8)


# bf16 rows of whole chunks that come through shared memory, with windows up to
# the widest: some leave the rows room there, some do not
@pytest.mark.parametrize("sk", [7168, 7176, 8192, 9224, 14344, 16384])
@pytest.mark.parametrize("buckets,far,two", [(256, 2048, True), (128, 2048, True), (64, 2048, True), (256, 1536, True),
                                             (128, 2048, False)])
def test_wide_windows_of_staged_rows(buckets, far, two, sk):
    x, dy, table, m = inputs(1, 2, 3, sk, BF, seed=22, buckets=buckets, mask="heads")
    kw = dict(table=table, max_distance=far, bidirectional=two, q_start=sk // 2)
    check(x, dy, **kw)
    check(x, dy, mask=m, causal=True, p=0.1, seed=9, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sk", [40, 300, 5000, 40000])
def test_masks_of_any_finite_value(sk, dtype):
    """Masks whose product with log2 e is beyond the type, up to its largest
    and down to its lowest, are added as exactly as others; so are scores well
    above 66 under an ordinary mask."""
    x, dy, table, _ = inputs(1, 2, 7, sk, dtype, seed=23)
    m = torch.zeros(1, 1, 7, sk, device=DEV, dtype=dtype)
    m[:, :, 0] = 3e38
    m[:, :, 1] = torch.finfo(dtype).max
    m[:, :, 2, sk // 2:] = 3e38
    m[:, :, 3, sk // 3] = 3e38  # next to zeros: this key alone
    m[:, :, 4, : sk // 2], m[:, :, 4, sk // 2:] = 2.5e38, torch.finfo(dtype).min
    m[:, :, 5, sk // 2:] = -math.inf
    x[:, :, 5] *= 100
    check(x, dy, table=table, mask=m)
    check(x, dy, table=table, mask=m, causal=True, bidirectional=False, q_start=sk - 7, p=0.1, seed=2)


# Sizes at which a team works on several rows one after another (more rows than
# the GPU holds teams): 8 or 16 lanes, a warp, several warps, long rows and rows
# of several register blocks; whole and ragged ones; sq no multiple of a step.
# (Per window sum that is at most 64 rows of up to 4 chunks.)
WALKS = [(2, 8, 2101, 40), (3, 8, 1333, 37), (2, 8, 1103, 264), (2, 6, 701, 515), (2, 4, 515, 1032), (3, 2, 333, 2051),
         (2, 4, 101, 9000), (2, 2, 151, 20008)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", WALKS)
def test_several_rows_a_team(size, dtype):
    b, np_, sq, sk = size
    x, dy, table, m = inputs(*size, dtype, seed=sk, mask="pad")
    check(x, dy, table=table, q_start=sk // 3)
    check(x, dy, table=table, mask=m, causal=True, bidirectional=False, q_start=sk - sq // 2, p=0.1, seed=3)
    starts = torch.tensor([7 * i - 3 for i in range(b)], dtype=torch.int32, device=DEV)
    y, _, dx, dt = run_both(x, dy, table=table, seq_start=starts, q_start=sk // 2, p=0.25, seed=4)
    for i in range(b):  # each batch alone, at its own position and elements
        kw = dict(table=table, q_start=sk // 2 + 7 * i - 3, p=0.25, seed=4, elem_base=i * np_ * sq * sk)
        yi, _, dxi, _ = run_both(x[i:i + 1].clone(), dy[i:i + 1].clone(), **kw)
        ry, ty, rdx, tdx, _, _ = reference(x[i:i + 1], 0.125, dy=dy[i:i + 1], **kw)
        for got in (y[i:i + 1], yi):
            close(got, ry, ty, "y")
        for got in (dx[i:i + 1], dxi):
            close(got, rdx, tdx, "dx")
