"""One encoder layer with expert MLPs, forward and backward, on libmfx.

The matrix products are torch's; everything between them is the library's:

  scores  -> mfx_relbias_softmax_dropout (learned relative position bias,
             padding mask, softmax and dropout in one pass)
  residual-> mfx_bias_dropout_add_train_nomask (the mask is drawn again by the
             backward, none is stored)
  experts -> mfx_moe_sort, mfx_moe_permute (tokens and their weights by
             expert), mfx_bias_swiglu with a weight per row, mfx_moe_unpermute

Run it on a GPU:  python examples/expert_layer.py
"""
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import elementwise_epilogues_transformer_gb300 as mfx  # noqa: E402


@dataclass
class Sizes:
    batch: int = 4
    seq: int = 1024
    heads: int = 16
    head_dim: int = 64
    experts: int = 8
    topk: int = 2
    ffn: int = 2048
    buckets: int = 32
    max_distance: int = 128
    p: float = 0.1

    @property
    def hidden(self):
        return self.heads * self.head_dim


def make_params(c, dtype, device="cuda", seed=0):
    g = torch.Generator().manual_seed(seed)
    new = lambda *s, std: (torch.randn(s, generator=g) * std).to(dtype).to(device)  # noqa: E731
    h, f, std = c.hidden, c.ffn, c.hidden ** -0.5
    return {"wq": new(h, h, std=std), "wk": new(h, h, std=std), "wv": new(h, h, std=std), "wo": new(h, h, std=std),
            "table": new(c.buckets, c.heads, std=0.5), "bo": new(h, std=0.02), "wr": new(h, c.experts, std=std),
            "w1": new(c.experts, h, 2 * f, std=std), "w2": new(c.experts, f, h, std=f ** -0.5), "b2": new(h, std=0.02)}


class ExpertLayer:
    """forward() keeps what backward() needs; backward() returns (dx, grads)."""

    def __init__(self, sizes, params, seed=1234):
        self.c, self.w, self.seed = sizes, params, seed

    def _heads(self, t):
        return t.view(self.c.batch, self.c.seq, self.c.heads, self.c.head_dim).transpose(1, 2)

    def _tokens(self, t):
        return t.transpose(1, 2).reshape(self.c.batch * self.c.seq, self.c.hidden)

    def _by_expert(self, rows, weights, out, transpose=False):
        """out[rows of e] = rows[of e] @ weights[e] (or its transpose)."""
        for e, (a, b) in enumerate(zip(self.begin[:-1], self.begin[1:])):
            torch.matmul(rows[a:b], weights[e].t() if transpose else weights[e], out=out[a:b])
        out[self.begin[-1]:] = 0
        return out

    def forward(self, x, mask=None):
        c, w = self.c, self.w
        self.x, self.mask, self.scale = x, mask, c.head_dim ** -0.5
        # attention
        self.q, self.k, self.v = (self._heads(x @ w[n]) for n in ("wq", "wk", "wv"))
        self.scores = self.q @ self.k.transpose(2, 3)
        self.softmax = dict(table=w["table"], mask=mask, max_distance=c.max_distance, p=c.p, seed=self.seed, offset=0)
        self.probs, self.stats = mfx.mfx_relbias_softmax_dropout_fwd(self.scores, self.scale, **self.softmax)
        self.ctx = self._tokens(self.probs @ self.v)
        self.h = mfx.mfx_bias_dropout_add_train_nomask(self.ctx @ w["wo"], w["bo"], x, c.p, self.seed, offset=1)
        # the router: probabilities of the chosen experts, made to sum to one
        self.gates = (self.h.float() @ w["wr"].float()).softmax(-1)
        top, self.choice = self.gates.topk(c.topk, dim=-1)
        self.total = top.sum(-1, keepdim=True)
        self.weight = top / self.total
        # experts
        self.row_of, self.slot_of, offsets, _ = mfx.mfx_moe_sort(self.choice.int(), c.experts, align=8)
        self.begin = offsets.tolist()
        rows = self.slot_of.numel()
        new = lambda n: torch.empty((rows, n), dtype=x.dtype, device=x.device)  # noqa: E731
        self.hp, self.wp = mfx.mfx_moe_permute_fwd(self.h, self.row_of, self.slot_of, weight=self.weight)
        self.z = self._by_expert(self.hp, w["w1"], new(2 * c.ffn))
        self.a = mfx.mfx_bias_swiglu_fwd(self.z, None, self.wp)
        y = self._by_expert(self.a, w["w2"], new(c.hidden))
        out = mfx.mfx_moe_unpermute_fwd(y, self.row_of)
        return mfx.mfx_bias_dropout_add_train_nomask(out, w["b2"], self.h, c.p, self.seed, offset=2)

    def backward(self, g):
        c, w, d = self.c, self.w, {}
        # experts
        gout, gh, d["b2"] = mfx.mfx_bias_dropout_add_bwd_dbias(g, None, c.p, self.seed, 2, residual_dtype=g.dtype)
        gy, _ = mfx.mfx_moe_unpermute_bwd(gout, None, self.row_of, self.slot_of)
        d["w2"], d["w1"] = torch.empty_like(w["w2"]), torch.empty_like(w["w1"])
        ga = self._by_expert(gy, w["w2"], torch.empty_like(self.a), transpose=True)
        gz, gwp = mfx.mfx_bias_swiglu_bwd(ga, self.z, None, self.wp)
        ghp = self._by_expert(gz, w["w1"], torch.empty_like(self.hp), transpose=True)
        for e, (a, b) in enumerate(zip(self.begin[:-1], self.begin[1:])):
            torch.matmul(self.a[a:b].t(), gy[a:b], out=d["w2"][e])
            torch.matmul(self.hp[a:b].t(), gz[a:b], out=d["w1"][e])
        gh_experts, gweight = mfx.mfx_moe_permute_bwd(ghp, self.row_of, g_weight=gwp)
        # router
        gtop = (gweight - (gweight * self.weight).sum(-1, keepdim=True)) / self.total
        ggates = torch.zeros_like(self.gates).scatter_(-1, self.choice, gtop)
        glogits = self.gates * (ggates - (ggates * self.gates).sum(-1, keepdim=True))
        d["wr"] = (self.h.float().t() @ glogits).to(w["wr"].dtype)
        gh = gh + gh_experts + (glogits @ w["wr"].float().t()).to(g.dtype)
        # attention
        gattn, gx, d["bo"] = mfx.mfx_bias_dropout_add_bwd_dbias(gh, None, c.p, self.seed, 1, residual_dtype=g.dtype)
        d["wo"] = self.ctx.t() @ gattn
        gctx = self._heads(gattn @ w["wo"].t())
        gscores, d["table"] = mfx.mfx_relbias_softmax_dropout_bwd(
            gctx @ self.v.transpose(2, 3), self.scores, self.stats, self.scale, **self.softmax)
        for n, t in (("wq", gscores @ self.k), ("wk", gscores.transpose(2, 3) @ self.q),
                     ("wv", self.probs.transpose(2, 3) @ gctx)):
            t = self._tokens(t)
            d[n] = self.x.t() @ t
            gx = gx + t @ w[n].t()
        return gx, d


def main():
    c, dtype = Sizes(), torch.bfloat16
    layer = ExpertLayer(c, make_params(c, dtype))
    x = torch.randn(c.batch * c.seq, c.hidden, device="cuda").to(dtype)
    lengths = torch.randint(c.seq // 2, c.seq + 1, (c.batch,), device="cuda")
    mask = torch.where(torch.arange(c.seq, device="cuda") < lengths[:, None], 0.0, float("-inf"))
    mask = mask.to(dtype).view(c.batch, 1, 1, c.seq)
    for _ in range(3):
        dx, grads = layer.backward(layer.forward(x, mask))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    out = layer.forward(x, mask)
    dx, grads = layer.backward(torch.ones_like(out))
    end.record()
    torch.cuda.synchronize()
    finite = all(bool(torch.isfinite(t).all()) for t in (out, dx, *grads.values()))
    print(f"{c.batch * c.seq} tokens x {c.hidden}, {c.experts} experts: forward and backward "
          f"{begin.elapsed_time(end):.3f} ms, all values finite: {finite}")


if __name__ == "__main__":
    main()
