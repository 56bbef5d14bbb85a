"""The example layer, which runs the position bias, the dropouts without a mask
and the expert maps together, against torch's autograd over the plain form in
64 bits with the same keep flags.

A value passes at most some 25 fp32 operations whose sums have up to 128
terms, and the products of its backward again: 50 * 128 half steps of the
norm, 4e-4."""
import importlib.util
import os

import pytest
import torch

import elementwise_epilogues_transformer_gb300 as mfx
from relbias_ref import bucket, keep_flags

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
E = importlib.util.module_from_spec(spec)
spec.loader.exec_module(E)


def plain(c, w, x, mask, seed, choice):
    """The layer from its definition; the experts are those the layer chose."""
    n = c.batch * c.seq
    heads = lambda t: t.view(c.batch, c.seq, c.heads, c.head_dim).transpose(1, 2)
    drop = lambda t, offset: t * (keep_flags(t.shape, c.p, seed, offset, 0).to(t.device) / (1 - c.p))
    q, k, v = (heads(x @ w[m]) for m in ("wq", "wk", "wv"))
    pos = torch.arange(c.seq, device=x.device)
    bias = w["table"][bucket(pos[None] - pos[:, None], c.buckets, c.max_distance, True)].permute(2, 0, 1)
    s = q @ k.transpose(2, 3) * c.head_dim ** -0.5 + bias + mask.double()
    ctx = (drop(s.softmax(-1), 0) @ v).transpose(1, 2).reshape(n, c.hidden)
    h = drop(ctx @ w["wo"] + w["bo"], 1) + x
    gates = (h @ w["wr"]).softmax(-1)
    top = gates.gather(-1, choice)
    weight = top / top.sum(-1, keepdim=True)
    out = 0
    for e in range(c.experts):
        z = h @ w["w1"][e]
        y = (torch.nn.functional.silu(z[:, :c.ffn]) * z[:, c.ffn:]) @ w["w2"][e]
        out = out + y * (weight * (choice == e)).sum(-1, keepdim=True)
    return drop(out + w["b2"], 2) + h


@pytest.mark.parametrize("sizes", [E.Sizes(2, 33, 4, 16, 5, 2, 40), E.Sizes(3, 64, 2, 32, 4, 1, 24, buckets=8, p=0.3)])
def test_layer_against_autograd(sizes):
    c = sizes
    torch.backends.cuda.matmul.allow_tf32 = False
    params = E.make_params(c, torch.float32, seed=c.seq)
    g = torch.Generator().manual_seed(c.ffn)
    x, up = (torch.randn(c.batch * c.seq, c.hidden, generator=g).cuda() for _ in range(2))
    mask = torch.zeros(c.batch, 1, 1, c.seq, device="cuda")
    mask[0, ..., c.seq // 2:] = -float("inf")
    layer = E.ExpertLayer(c, params)
    out = layer.forward(x, mask)
    dx, grads = layer.backward(up)
    w64 = {k: v.double().requires_grad_() for k, v in params.items()}
    x64 = x.double().requires_grad_()
    want = plain(c, w64, x64, mask, layer.seed, layer.choice)
    want.backward(up.double())
    for name, a, b in [("out", out, want), ("dx", dx, x64.grad), *((k, grads[k], w64[k].grad) for k in grads)]:
        size = b.norm()
        if name == "wr" and c.topk == 1:
            # one choice: its weight is one whatever the router says, the gradient zero but for what cancels
            assert size <= 1e-12 * w64["w1"].grad.norm()
            size = w64["w1"].grad.norm()
        err = ((a.double() - b).norm() / size).item()
        assert err <= 4e-4, (name, err)
    assert mfx.mfx_device_error() == 0
