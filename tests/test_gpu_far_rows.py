"""Rows whose first element lies past 2^31 elements from the buffer's: the
distillation's calls, the norm's backward and its 8-bit form, and every row that
the log probabilities leave out."""
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import U, distill, distill_bwd, excess, half, norm_bwd, norm_fwd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
ROWS, COLS = 66000, 33000  # 2.18e9 elements
SOME = [0, 1, 32999, 65075, 65076, 65534, 65999]  # row 65076 is the first past 2^31


def data():
    t = torch.empty((ROWS, COLS), dtype=BF, device=DEV)
    t.normal_()
    return t


def others_are_zero(d, some):
    """All rows but `some`, a slice at a time."""
    keep = torch.ones(ROWS, dtype=torch.bool, device=DEV)
    keep[some] = False
    for at in range(0, ROWS, 4096):
        assert not d[at:at + 4096].ne(0).any(1)[keep[at:at + 4096]].any(), at


@pytest.mark.parametrize("form", ["apart", "apart in place", "one call", "one call in place"])
def test_distill(form):
    torch.manual_seed(4)
    z, some = data(), torch.tensor(SOME, device=DEV)
    index = torch.full((ROWS, 3), -1, dtype=torch.int64, device=DEV)
    index[some] = torch.randint(0, COLS, (len(SOME), 3), device=DEV)
    index[some[-1], 2] = COLS - 1
    teacher, g = torch.randn((ROWS, 3), device=DEV), torch.rand(ROWS, device=DEV)
    r, q, want, tol, q_tol = distill(z[some], index[some], teacher[some], 1.0)
    d_want, d_tol = distill_bwd(r, q, q_tol, index[some], g[some], 1.0, COLS)
    out = z if form.endswith("in place") else None
    if form.startswith("apart"):
        loss, stats = mfx.mfx_topk_distill_fwd(z, index, teacher)
        d = mfx.mfx_topk_distill_bwd(g, z, index, teacher, stats, dlogits=out)
    else:
        loss, d = mfx.mfx_topk_distill_fwd_bwd(z, index, teacher, g, dlogits=out)
    assert excess(loss[some], want, tol) <= 1 and int((loss != 0).sum()) == len(SOME)
    assert excess(d[some], d_want, d_tol + d_want.abs() * half(BF)) <= 1
    others_are_zero(d, some)


def test_logprobs_rows_left_out():
    torch.manual_seed(5)
    z, some = data(), torch.tensor(SOME, device=DEV)
    tokens = torch.full((ROWS,), -1, dtype=torch.int32, device=DEV)
    tokens[some] = 7
    stats = mfx.mfx_token_logprobs_fwd(z, tokens)[4]
    g = torch.ones(ROWS, device=DEV)
    d = mfx.mfx_token_logprobs_bwd(g, None, z, tokens, stats, dlogits=z)
    assert (d[some, 7] > 0).all()
    others_are_zero(d, some)


@pytest.mark.parametrize("cols", [4096, 33000])
def test_norm(cols):
    """Backward and 8 bits, a row in a block and a row that is read twice."""
    torch.manual_seed(6)
    rows = (1 << 31) // cols + 300
    some = torch.tensor([0, 1, rows // 2, (1 << 31) // cols, (1 << 31) // cols + 1, rows - 1], device=DEV)
    h = torch.empty((rows, cols), dtype=BF, device=DEV)
    h.normal_()
    w = torch.rand(cols, device=DEV) + 0.5
    q, scale, _, rstd = mfx.mfx_add_rmsnorm_quant_fwd(h, w, group=128, need_rstd=True)
    _, y, r, rel = norm_fwd(h[some], None, w, 1e-6, 0.0)
    s = scale[some].double().repeat_interleave(128, 1)[:, :cols]
    assert excess(rstd[some], r, r * rel) <= 1
    assert excess(q.view(torch.uint8)[some].view(q.dtype).double() * s, y, y.abs() * (2.0 ** -4 + 2 * rel + 8 * U) + s * 2.0 ** -10 * (1 + 1e-6)) <= 1
    del q, scale
    dy = torch.zeros_like(h)  # the rows that are looked at have a gradient, so the sum over rows is theirs
    dy[some] = torch.randn((some.numel(), cols), device=DEV).to(BF)
    d, tol, dw, dw_tol = norm_bwd(dy[some], h[some], rstd[some], w, None, 0.0)
    dx, _, dweight = mfx.mfx_add_rmsnorm_bwd(dy, h, rstd, w, dx=dy)
    assert excess(dx[some], d, tol + d.abs() * half(BF)) <= 1
    assert excess(dweight, dw, dw_tol + dw.abs() * half(F32)) <= 1
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[some] = False
    for at in range(0, rows, 65536):
        assert not dx[at:at + 65536].ne(0).any(1)[keep[at:at + 65536]].any(), at
