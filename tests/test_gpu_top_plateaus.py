"""Alternatives of very long rows with plateaus of equal logits that begin
late: the search meets more candidates than it has room for when it has taken
part of its threads' runs already."""
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import top_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"


def plateaus(vocab, dtype, period, starts, few):
    """Rows of -1 to -2 with zeros from `start` on of every `period` columns,
    and a few larger logits before the first zeros of each period."""
    place = torch.arange(vocab, device=DEV) % period
    rows = []
    for start in starts:
        z = torch.where(place < start, -1.0 - torch.rand(vocab, device=DEV), 0.0)
        for n in few:
            y = z.clone()
            y[torch.randint(0, start, (n,), device=DEV)] = torch.randint(1, 9, (n,), device=DEV).float()
            rows.append(y)
    z = rows[0].clone()
    z[32:64:8] = 2.0  # the first group of threads or parts
    rows.append(z)
    return torch.stack(rows).to(dtype)


def check(z, copies, tops):
    want = top_of(z, torch.ones(z.shape[0], dtype=torch.bool, device=DEV), max(tops))
    many = z.repeat(copies, 1)
    tokens = torch.zeros(many.shape[0], dtype=torch.int32, device=DEV)
    for top in tops:
        _, _, value, index, _ = mfx.mfx_token_logprobs_fwd(many, tokens, top=top, need_stats=False)
        index = index.view(copies, z.shape[0], top)
        for i in range(copies):
            assert torch.equal(index[i].long(), want[:, :top]), (top, i)
        assert torch.equal(value[:, :-1] >= value[:, 1:], torch.ones_like(value[:, 1:], dtype=torch.bool))


# slices of 125 000 columns, a thread's first 32 runs 32768 (fp32) or 65536 (bf16) of them
@pytest.mark.parametrize("vocab,dtype,period", [(1_000_000, F32, 125_000), (1_000_003, F32, 125_001), (600_000, F32, 75_000),
                                                (2_000_000, BF, 250_000), (1_200_007, BF, 150_001)])
def test_few_rows(vocab, dtype, period):
    torch.manual_seed(7)
    z = plateaus(vocab, dtype, period, [period // 4, period // 3, period // 2, period - 3000], (0, 3, 19, 60, 100))
    check(z, 1, (1, 5, 24, 25, 64))


# a part's first 16 runs are 32768 columns (bf16) of 65536 or more
@pytest.mark.parametrize("vocab,dtype,period", [(500_000, BF, 65_536), (500_009, BF, 65_536), (800_000, BF, 106_496),
                                                (300_000, F32, 40_960)])
def test_many_rows(vocab, dtype, period):
    torch.manual_seed(8)
    z = plateaus(vocab, dtype, period, [period // 2, period // 2 + 5000, period - 9000], (0, 3, 10, 60, 100))
    check(z, 20, (1, 20, 24, 25, 64))
