"""Dropout whose mask is never stored: bit for bit what the oracle's and the
mask-writing call's keep flags say."""
import numpy as np
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
import oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def flags(n, p, seed, offset, base):
    z = np.zeros((1, n), np.float32)
    return torch.from_numpy(O.bias_dropout_add_train(z, z, None, p=p, seed=seed, offset=offset, elem_base=base)[1]).view(
        -1).bool()


def shifted(t, k):
    buf = torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)
    v = buf[k:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 2048, 4099, 70001, 300000])
@pytest.mark.parametrize("base", [0, 3, 8 * (1 << 33), 12345678901])
def test_plain(n, base, dtype):
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype).to(DEV)
    for p in (0.0, 0.1, 0.5):
        scale = torch.tensor(1.0) / (torch.tensor(1.0) - torch.tensor(p))
        want = torch.where(flags(n, p, 77, 5, base).to(DEV), (x.float() * scale.to(DEV)).to(dtype), torch.zeros_like(x))
        for k in (0, 1, 4):
            v = shifted(x, k)
            assert torch.equal(mfx.mfx_dropout_fwd(v, p, 77, 5, base), want)
            assert torch.equal(mfx.mfx_dropout_bwd(v, p, 77, 5, base, dx=v), want)  # in place


@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (64, 1024), (33, 4099), (129, 640)])
@pytest.mark.parametrize("base", [0, 5])
def test_residual(rows, cols, base, dtype, res):
    """The bits of the mask-writing call, and its backward from the regenerated mask."""
    g = torch.Generator().manual_seed(rows + cols)
    new = lambda *s: torch.randn(s, generator=g)
    x, b, r, up = (new(rows, cols).to(dtype).to(DEV), new(cols).to(dtype).to(DEV), new(rows, cols).to(res).to(DEV),
                   new(rows, cols).to(dtype).to(DEV))
    key = (0.25, 99, 3, base)
    for bias in (b, None):
        want, mask = mfx.mfx_bias_dropout_add_train(x, bias, r, *key)
        for k in (0, 1):
            got = mfx.mfx_bias_dropout_add_train_nomask(shifted(x, k), bias, shifted(r, k), *key)
            assert torch.equal(got, want)
        y = x.clone()
        assert torch.equal(mfx.mfx_bias_dropout_add_train_nomask(y, bias, r, *key, out=y), want)
    for k in (0, 1):
        got = mfx.mfx_bias_dropout_add_bwd(shifted(up, k), None, *key, residual_dtype=res)
        for a, c in zip(got, mfx.mfx_bias_dropout_add_bwd(up, mask, *key, residual_dtype=res)):
            assert torch.equal(a, c)


def test_parts_of_a_tensor_share_its_mask():
    x = torch.randn(5000, device=DEV)
    whole = mfx.mfx_dropout_fwd(x, 0.3, 8)
    for a, b in ((0, 1), (1, 800), (800, 5000)):
        assert torch.equal(mfx.mfx_dropout_fwd(x[a:b].clone(), 0.3, 8, elem_base=a), whole[a:b])


def test_hidden_values():
    """What is dropped is zero whatever it was; what is kept keeps its NaN."""
    x = torch.full((4096,), float("nan"), device=DEV)
    keep = flags(4096, 0.5, 1, 0, 0).to(DEV)
    y = mfx.mfx_dropout_fwd(x, 0.5, 1)
    assert torch.isnan(y[keep]).all() and not y[~keep].any()


def test_empty_and_large_offsets():
    assert mfx.mfx_dropout_fwd(torch.empty(0, 4, device=DEV), 0.1, 1).shape == (0, 4)
    with pytest.raises(mfx.MfxError):
        mfx.mfx_dropout_fwd(torch.empty(16, device=DEV), 0.1, 1, elem_base=2 ** 64 - 8)
    with pytest.raises(mfx.MfxError):
        mfx.mfx_dropout_fwd(torch.empty(16, device=DEV), 1.0, 1)


def test_graph_and_stream():
    x = torch.randn(1000, 333, device=DEV, dtype=BF)
    want = mfx.mfx_dropout_fwd(x, 0.1, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mfx.mfx_dropout_fwd(x, 0.1, 4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mfx.mfx_dropout_fwd(x, 0.1, 4, out=out)
    g.replay()
    assert torch.equal(out, want)


# several units a lane (from 1.2 million fp32 or 2.5 million bf16 elements on), and one beside it
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [5, 4099, 1_000_003, 3_100_005])
@pytest.mark.parametrize("base", [0, 5, 12345678901])
def test_every_alignment(n, base, dtype):
    """Input and output any number of elements off a vector, alike or not, at
    element offsets on and off a generator block."""
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dtype).to(DEV)
    p = 0.25
    scale = torch.tensor(1.0) / (torch.tensor(1.0) - torch.tensor(p))
    want = torch.where(flags(n, p, 77, 5, base).to(DEV), (x.float() * scale.to(DEV)).to(dtype), torch.zeros_like(x))
    for a in (0, 1, 3, 4, 7):
        v = shifted(x, a)
        for b in (0, 1, 4, 6):
            out = shifted(torch.full_like(x, float("nan")), b)
            assert torch.equal(mfx.mfx_dropout_fwd(v, p, 77, 5, base, out=out), want), (a, b)
        assert torch.equal(mfx.mfx_dropout_bwd(v, p, 77, 5, base, dx=v), want), a


@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", [(7, 333), (1033, 3001), (1024, 4096)])
@pytest.mark.parametrize("base", [0, 5])
def test_regenerated_backward_at_every_alignment(rows, cols, base, dtype, res):
    """dx and dresidual are the bits of the backward that reads the mask."""
    g = torch.Generator().manual_seed(rows)
    x, up = (torch.randn(rows, cols, generator=g).to(dtype).to(DEV) for _ in range(2))
    key = (0.25, 99, 3, base)
    _, mask = mfx.mfx_bias_dropout_add_train(x, None, x, *key)
    want = mfx.mfx_bias_dropout_add_bwd(up, mask, *key, residual_dtype=res)
    for a, b, c in ((0, 0, 0), (1, 1, 1), (1, 0, 0), (0, 3, 1), (4, 4, 4), (5, 2, 0), (0, 0, 2)):
        dx = shifted(torch.full_like(up, float("nan")), b)
        dres = shifted(torch.full((rows, cols), float("nan"), dtype=res, device=DEV), c)
        got = mfx.mfx_bias_dropout_add_bwd(shifted(up, a), None, *key, dx=dx, dresidual=dres)
        for i in range(2):
            assert torch.equal(got[i], want[i]), (a, b, c, i)
