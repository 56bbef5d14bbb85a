"""Calls on another stream than the current one: what they allocate for
themselves must not be given to the current stream while they have yet to run."""
import numpy as np
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx

pytestmark = pytest.mark.gpu

DEV = "cuda"


def calls(stream):
    """Outputs of the operators that allocate, with workspaces of their own among them."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 4, 64, 512, generator=g).bfloat16().to(DEV)
    table = torch.randn(32, 4, generator=g).to(DEV)
    chosen = torch.randint(0, 16, (3000, 4), generator=g, dtype=torch.int32).to(DEV)
    tokens = torch.randn(3000, 256, generator=g).bfloat16().to(DEV)
    weight = torch.rand(3000, 4, generator=g).to(DEV)
    bias = torch.randn(256, generator=g).bfloat16().to(DEV)
    torch.cuda.synchronize()

    def run():
        kw = dict(table=table, p=0.1, seed=3, stream=stream)
        y, stats = mfx.mfx_relbias_softmax_dropout_fwd(x, 0.125, **kw)
        dx, dtable = mfx.mfx_relbias_softmax_dropout_bwd(y, x, stats, 0.125, **kw)
        row_of, slot_of, ends, counts = mfx.mfx_moe_sort(chosen, 16, align=8, stream=stream)
        rows, _ = mfx.mfx_moe_permute_fwd(tokens, row_of, slot_of, stream=stream)
        out = mfx.mfx_moe_unpermute_fwd(rows, row_of, weight, stream=stream)
        dy, dweight = mfx.mfx_moe_unpermute_bwd(out, rows, row_of, slot_of, weight, stream=stream)
        dtokens, _ = mfx.mfx_moe_permute_bwd(dy, row_of, stream=stream)
        add = mfx.mfx_bias_dropout_add_train_nomask(tokens, bias, out, 0.1, 3, stream=stream)
        drop = mfx.mfx_dropout_bwd(mfx.mfx_dropout_fwd(tokens, 0.1, 3, stream=stream), 0.1, 3, stream=stream)
        _, dbias = mfx.mfx_bias_gelu_bwd_dbias(tokens, bias, tokens, stream=stream)
        return [y, stats, dx, dtable, row_of, slot_of, ends, counts, rows, out, dy, dweight, dtokens, add, drop, dbias]

    return run


@pytest.mark.parametrize("kind", ["stream", "handle", "default"])
def test_other_stream(kind):
    want = calls(None)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = {"stream": side, "handle": side.cuda_stream, "default": 0}[kind]
    run = calls(stream)
    here = torch.cuda.current_stream() if kind != "default" else side
    other = side if kind != "default" else torch.cuda.default_stream()
    with torch.cuda.stream(here):
        with torch.cuda.stream(other):
            torch.cuda._sleep(20_000_000)  # about 10 ms: the calls wait in line
        got = run()
        # whatever memory is free to this stream is written at once
        for shift in range(9, 24):
            for _ in range(4):
                torch.empty(1 << shift, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_empty_workspace():
    """An empty workspace, whose pointer is null, is not taken for a question
    about the size: it is refused, or does where none is needed."""
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    x = torch.randn(2, 3, 4, 64, device=DEV)
    table = torch.randn(32, 3, device=DEV)
    y, stats = mfx.mfx_relbias_softmax_dropout_fwd(x, 0.125, table=table)
    chosen = torch.arange(8000, dtype=torch.int32, device=DEV).view(2000, 4) % 16
    g, b = x.view(24, 64), torch.zeros(64, device=DEV)
    for call in (lambda ws: mfx.mfx_relbias_softmax_dropout_bwd(y, x, stats, 0.125, table=table, workspace=ws),
                 lambda ws: mfx.mfx_moe_sort(chosen, 16, workspace=ws),
                 lambda ws: mfx.mfx_bias_gelu_bwd_dbias(g, b, g, workspace=ws),
                 lambda ws: mfx.mfx_bias_dropout_add_bwd_dbias(g, None, 0.1, 1, workspace=ws)):
        for ws in (none, lambda n: none):
            with pytest.raises(mfx.MfxError) as e:
                call(ws)
            assert e.value.status == 8
    few = chosen[:100].contiguous()
    maps = [torch.full(s, -7, dtype=torch.int32, device=DEV) for s in ((100, 4), (400,), (17,), (16,))]
    got = mfx.mfx_moe_sort(few, 16, workspace=none, **dict(zip(("row_of", "slot_of", "offsets", "counts"), maps)))
    for a, c in zip(got, mfx.mfx_moe_sort(few, 16)):
        assert torch.equal(a, c)


def test_numbers_of_other_kinds():
    """Scalars from numpy and 0-dim tensors count as the numbers that they are, as in the other calls."""
    x = torch.randn(2, 3, 4, 64, device=DEV)
    table = torch.randn(32, 3, device=DEV)
    kw = dict(table=table, max_distance=100, q_start=20, p=0.25, seed=2**63 + 5, offset=3, elem_base=8)
    i, f = np.int64, np.float64
    other = dict(table=table, max_distance=i(100), q_start=i(20), p=f(0.25), seed=np.uint64(2**63 + 5), offset=i(3),
                 elem_base=torch.tensor(8))
    y, stats = mfx.mfx_relbias_softmax_dropout_fwd(x, 0.125, **kw)
    y2, stats2 = mfx.mfx_relbias_softmax_dropout_fwd(x, torch.tensor(0.125), **other)
    assert torch.equal(y, y2) and torch.equal(stats, stats2)
    for a, b in zip(mfx.mfx_relbias_softmax_dropout_bwd(y, x, stats, 0.125, **kw),
                    mfx.mfx_relbias_softmax_dropout_bwd(y, x, stats, np.float32(0.125), **other)):
        assert torch.equal(a, b)
    chosen = torch.arange(400, dtype=torch.int32, device=DEV).view(100, 4) % 16
    for a, b in zip(mfx.mfx_moe_sort(chosen, 16, align=8, capacity=20, rows=600),
                    mfx.mfx_moe_sort(chosen, torch.tensor(16), align=i(8), capacity=i(20), rows=i(600))):
        assert torch.equal(a, b)
    assert mfx.mfx_moe_rows(i(10), i(2), i(4), i(16)) == 80
