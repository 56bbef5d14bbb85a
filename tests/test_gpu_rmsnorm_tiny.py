"""The norm in 8 bits where values are so small that a scale's reciprocal and
rstd together pass fp32's range: zeros stay zeros, nothing saturates."""
import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from vocab_ref import U, excess, norm_fwd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
DEV = "cuda:0"


def check(x, weight, group, qdt, sdt):
    cols = x.shape[-1]
    q, scale, _, rstd = mfx.mfx_add_rmsnorm_quant_fwd(x, weight, group=group, q_dtype=qdt, scale_dtype=sdt, need_rstd=True)
    _, y, r, rel = norm_fwd(x, None, weight, 1e-6, 0.0)
    assert excess(rstd, r, r * rel) <= 1
    n = group or cols
    tops = torch.stack([p.abs().max(1).values for p in y.split(n, 1)], 1)
    ideal = torch.where(tops == 0, 1.0, (tops / torch.finfo(qdt).max).clamp(min=2.0 ** -126))
    # products below 2^-126 are off by half of 2^-149, before the factor rstd
    low = 2.0 ** -149 * r[:, None]
    s = scale.double()
    if sdt is E8:
        assert (s * (1 + 3 * rel) + low >= ideal).all() and (s < 2 * ideal * (1 + 3 * rel) + low).all()
    else:
        assert excess(scale, ideal, ideal * (rel + 4 * U) + low) <= 1
    # half a step of the type, or of its smallest numbers
    step, least = torch.finfo(qdt).eps / 2, torch.finfo(qdt).smallest_normal * torch.finfo(qdt).eps / 2
    s = s.repeat_interleave(n, 1)[:, :cols]
    assert excess(q.double() * s, y, y.abs() * (step + 2 * rel + 8 * U) + s * least * (1 + 1e-6) + 2 * low) <= 1
    assert q.float()[y == 0].eq(0).all()


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("qdt,sdt", [(E4, F32), (E4, E8), (E5, F32), (E5, E8)])
@pytest.mark.parametrize("cols", [40, 264, 520, 1000, 2051, 4096, 8192, 8200, 16384, 20001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tiny(cols, qdt, sdt, group, dtype):
    x = torch.randn((7, cols), device=DEV)
    x[:, ::3] = 0.0
    x *= torch.tensor([1.0, 1e-33, 1e-35, 1e-36, 1e-37, 0.1, 0.0], device=DEV)[:, None]
    check(x.to(dtype), torch.rand(cols, device=DEV) + 0.5, group, qdt, sdt)
    # weights that have died away: some groups', and all
    w = torch.rand(cols, device=DEV) + 0.5
    w[:min(cols, 256)] *= 1e-37
    x = torch.randn((7, cols), device=DEV) * torch.tensor([1.0, 0.2, 0.1, 0.03, 1e-3, 10.0, 0.0], device=DEV)[:, None]
    x[:, ::5] = 0.0
    for weight in (w, torch.full_like(w, 1e-37), torch.full_like(w, 3e-36)):
        check(x.to(dtype), weight, group, qdt, sdt)
