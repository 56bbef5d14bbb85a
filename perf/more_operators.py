"""Measured cases of three operators at a model's output: the root-mean-square norm with the residual's addition (plain
or with an output in 8 bits), log probabilities of given tokens with entropy and top alternatives, and distillation
from a teacher's top logits.

``run`` computes them in their plain form (elementary torch operations in 32 bits, 64 for long sums and next to the
borders of 8-bit types), or through the package's entry points where ``own`` is true.  ``exact`` is the same from the
definitions in 64 bits.

Definitions (rows are tokens):

* norm: h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * (weight + offset).  h is kept in the
  residual's type for the next layer and the backward.  In 8 bits, each group of a row's columns (the whole row, 128 or
  32 of them) has the scale s = max|y| / largest (448 for e4m3, 57344 for e5m2; 1 for a group of zeros, at least
  2^-126), as 32 bits or rounded up to a power of two, and q = y / s.  Backward, from the stored h: n = h * rstd,
  u = dy * (weight + offset), dx = rstd * (u - n * mean(u * n)) + dh, dweight = sum over rows of dy * n.
* logprobs: p = softmax(scale * z); logprob = log p[token], entropy = -sum p log p, and the `top` largest logits'
  log probabilities and columns, ties by the lowest column, (-inf, -1) where fewer are above -inf.  Rows whose token
  is negative are left out: zeros, (-inf, -1), no gradient.  dz = scale * (g * (1[token] - p) - ge * p * (log p +
  entropy)).
* distill: q = softmax(scale * t) over a row's teacher logits t (or exp(scale * t - lse) where the teacher's own lse
  is given), at columns `index`; negative columns hold nothing.  loss = sum q (log q - log p[index]);
  dz = g * scale * (sum(q) p - q at its columns).
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, rows, cols, dtype, residual, step, weight="bf16", offset=0.0, quant="none", group=0, scales="fp32"):
    c = dict(op="norm", rows=rows, cols=cols, dtype=dtype, residual=residual, step=step, weight=weight, offset=offset,
             quant=quant, group=group, scales=scales)
    return dict(c, name=name) if name else c


def _logprobs(name, rows, vocab, dtype, step, top=0, scale=1.0, pad=0, masked=0.0, lost=0.0):
    c = dict(op="logprobs", rows=rows, vocab=vocab, dtype=dtype, step=step, top=top, scale=scale, pad=pad,
             masked=masked, lost=lost)
    return dict(c, name=name) if name else c


def _distill(name, rows, vocab, k, dtype, step, teacher="bf16", scale=1.0, pad=0, lse=False, lost=0.0):
    c = dict(op="distill", rows=rows, vocab=vocab, k=k, dtype=dtype, step=step, teacher=teacher, scale=scale, pad=pad,
             lse=lse, lost=lost)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the norm before a block, forward and backward, on an fp32 residual stream
        _norm("norm train 16384x4096", 16384, 4096, "bf16", "fp32", "train"),
        # the same in a small fp32 model of an odd width, weights around zero
        _norm("norm train odd fp32 3001x2051", 3001, 2051, "fp32", "fp32", "train", weight="fp32", offset=1.0),
        # a prompt's norm before a product in 8 bits, a scale per token
        _norm("norm e4m3 rows 8192x8192", 8192, 8192, "bf16", "bf16", "infer", quant="e4m3"),
        # the same with a power of two per 32 columns
        _norm("norm e4m3 blocks 16384x4096", 16384, 4096, "bf16", "bf16", "infer", quant="e4m3", group=32,
              scales="e8m0"),
        # a decode batch, a scale per 128 columns
        _norm("norm e4m3 decode 32x8192", 32, 8192, "bf16", "bf16", "infer", quant="e4m3", group=128),
        # one new token: latency
        _norm("norm decode 1x4096", 1, 4096, "bf16", "bf16", "infer"),
        # a policy's log probabilities and entropy with their gradients
        _logprobs("logprobs train 8192x32768", 8192, 32768, "bf16", "train", lost=0.1),
        # a prompt scored with its alternatives, a large vocabulary
        _logprobs("logprobs top 1024x131072", 1024, 131072, "bf16", "infer", top=20),
        # one new token of a few sequences, with alternatives
        _logprobs("logprobs decode 8x131072", 8, 131072, "bf16", "infer", top=5, scale=1.25),
        # fp32 logits of an odd vocabulary within padded rows, some columns masked, with gradients
        _logprobs("logprobs odd fp32 333x50021", 333, 50021, "fp32", "train", top=3, pad=27, masked=0.1),
        # distillation with its gradient, the weight of each token known before
        _distill("distill 4096x131072 top 64", 4096, 131072, 64, "bf16", "fused", scale=0.5),
        # its forward and backward apart, odd sizes, the teacher's own normalisation
        _distill("distill apart odd 1001x32003", 1001, 32003, 16, "bf16", "apart", teacher="fp32", lse=True, lost=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "logprobs", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "norm":
        cols = rng.choice([1024, 4096, 8192, _log(rng, 64, 16384), _log(rng, 64, 16384)])
        rows = max(1, min(_log(rng, 1, 32768), (1 << 26) // cols))
        residual = rng.choice(["none", "bf16", "fp32"]) if dtype == "bf16" else rng.choice(["none", "fp32"])
        weight = rng.choice([dtype, "fp32"])
        offset = rng.choice([0.0, 1.0])
        if rng.random() < 0.5:
            return _norm(None, rows, cols, dtype, residual, rng.choice(["train", "train", "infer"]), weight, offset)
        group = rng.choice([0, 32, 128])
        return _norm(None, rows, cols, dtype, residual, "infer", weight, offset, rng.choice(["e4m3", "e4m3", "e5m2"]),
                     group, rng.choice(["fp32", "e8m0"]) if group else "fp32")
    vocab = rng.choice([32768, 131072, _log(rng, 128, 262144), _log(rng, 128, 262144)])
    rows = max(1, min(_log(rng, 1, 16384), (1 << 28) // vocab))
    pad = rng.choice([0, 0, rng.randint(1, 64)])
    scale = rng.choice([1.0, 0.5, rng.uniform(0.3, 2.0)])
    if kind == "logprobs":
        return _logprobs(None, rows, vocab, dtype, rng.choice(["train", "infer"]), rng.choice([0, 1, 5, 20, 64]), scale,
                         pad, rng.choice([0.0, 0.0, 0.5]), rng.choice([0.0, 0.1]))
    return _distill(None, rows, vocab, min(vocab // 2, _log(rng, 1, 256)), dtype, rng.choice(["fused", "apart"]),
                    rng.choice(["bf16", "fp32"]), scale, pad, rng.random() < 0.5, rng.choice([0.0, 0.1]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _rand(g, shape):
    return torch.rand(shape, generator=g, device="cuda")


def _logits(g, c):
    """A model's logits: most near each other, a few columns of each row far above."""
    rows, vocab = c["rows"], c["vocab"]
    z = _normal(g, (rows, vocab + c["pad"]), DT[c["dtype"]], 2.0)
    liked = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda")
    liked = (liked + torch.arange(8, device="cuda") * (vocab // 8)) % vocab
    z.scatter_(1, liked, _normal(g, liked.shape, z.dtype, 3.0) + 8)
    return z[:, :vocab], liked


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    rows = c["rows"]
    if c["op"] == "norm":
        shape, dt = (rows, c["cols"]), DT[c["dtype"]]
        s["x"] = _normal(g, shape, dt)
        # a residual stream: larger than what a block adds, some of its columns much larger
        s["residual"] = None
        if c["residual"] != "none":
            spread = torch.exp(torch.randn((c["cols"],), generator=g, device="cuda"))
            s["residual"] = (torch.randn(shape, generator=g, device="cuda") * spread).to(DT[c["residual"]])
        s["weight"] = (_normal(g, (c["cols"],), torch.float32, 0.2) + (1 - c["offset"])).to(DT[c["weight"]])
        if c["step"] == "train":
            s["dy"] = _normal(g, shape, dt)
            s["dh"] = None if s["residual"] is None else _normal(g, shape, DT[c["residual"]])
        return s
    s["logits"], liked = _logits(g, c)
    if c["op"] == "logprobs":
        if c["masked"]:  # columns that a grammar rules out
            s["logits"].masked_fill_(_rand(g, (1, c["vocab"])) < c["masked"], -math.inf)
        anywhere = torch.randint(0, c["vocab"], (rows,), generator=g, device="cuda")
        s["tokens"] = torch.where(_rand(g, (rows,)) < 0.8, liked[:, 0], anywhere)
        # a token that was sampled is not one that is ruled out: if it is, another row's column stands for it
        open_ = torch.isfinite(s["logits"].gather(1, s["tokens"][:, None])[:, 0])
        s["tokens"] = torch.where(open_, s["tokens"], s["logits"][:, :].argmax(1))
        s["tokens"] = torch.where(_rand(g, (rows,)) < c["lost"], -100, s["tokens"])
        if c["step"] == "train":
            s["g"], s["ge"] = _normal(g, (rows,), torch.float32), _normal(g, (rows,), torch.float32, 0.1)
        return s
    # the teacher likes much what the student likes
    near = s["logits"].float() + torch.randn(s["logits"].shape, generator=g, device="cuda")
    t, index = torch.topk(near, c["k"], dim=1)
    s["teacher"], s["index"] = t.to(DT[c["teacher"]]), index
    s["lse"] = torch.logsumexp(near * c["scale"], 1) if c["lse"] else None
    if c["lost"]:  # shorter lists, some of them empty
        length = torch.randint(0, c["k"] + 1, (rows, 1), generator=g, device="cuda")
        length = torch.where(_rand(g, (rows, 1)) < c["lost"], length, c["k"])
        s["index"] = torch.where(torch.arange(c["k"], device="cuda") < length, index, -1)
    s["g"] = _rand(g, (rows,)) / rows
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_quantised(c, y):
    """(q, scales) of y [rows, cols] in 64 bits."""
    rows, cols = y.shape
    n = c["group"] or cols
    groups = -(-cols // n)
    y = torch.cat([y, y.new_zeros((rows, groups * n - cols))], 1).view(rows, groups, n)
    top = y.abs().amax(2)
    s = (top / LARGEST[c["quant"]]).float().clamp(min=2.0 ** -126)
    if c["scales"] == "e8m0":
        part, power = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), power - (part == 0.5).int())
    s = torch.where(top == 0, 1.0, s)
    q = (y / s[..., None].double()).clamp(-LARGEST[c["quant"]], LARGEST[c["quant"]]).float().to(DT[c["quant"]])
    return q.view(rows, -1)[:, :cols].contiguous(), s.to(torch.float8_e8m0fnu) if c["scales"] == "e8m0" else s


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    w = s["weight"].float() + c["offset"]
    o = {} if s["residual"] is None else {"h": h.to(s["residual"].dtype)}
    if c["quant"] != "none":
        h = h.double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w.double()
        o["q"], o["scale"] = _plain_quantised(c, y)
        return o
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    o["y"] = (h * rstd * w).to(s["x"].dtype)
    if c["step"] == "train":
        n = (o["h"] if s["residual"] is not None else s["x"]).float() * rstd
        dy = s["dy"].float()
        u = dy * w
        d = rstd * (u - n * (u * n).mean(1, keepdim=True))
        if s["residual"] is not None:
            d = d + s["dh"].float()
            o["dresidual"] = d.to(s["residual"].dtype)
        o["dx"] = d.to(s["x"].dtype)
        o["dweight"] = (dy * n).sum(0, dtype=torch.float64).to(s["weight"].dtype)
    return o


def _plain_softmax(s):
    """(shifted scores, log of their powers' sum) of the logits' rows."""
    t = s["logits"].float()
    top = t.amax(1, keepdim=True)
    t = (t - torch.where(top == -math.inf, 0.0, top)) * s["case"]["scale"]
    return t, torch.log(torch.exp(t).sum(1, keepdim=True))


def _plain_logprobs(s):
    c = s["case"]
    kept = s["tokens"] >= 0
    token = s["tokens"].clamp(min=0)[:, None]
    t, log_sum = _plain_softmax(s)
    logp = t - log_sum
    p = torch.exp(logp)
    plogp = torch.where(p == 0, 0.0, p * logp)
    entropy = -plogp.sum(1, keepdim=True)
    o = {"logprob": torch.where(kept, logp.gather(1, token)[:, 0], 0.0),
         "entropy": torch.where(kept, entropy[:, 0], 0.0)}
    if c["top"]:
        # unique keys: the value's bits in their order, then the lowest column
        bits = (s["logits"].float() + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
        key = (order << 32) | (0xFFFFFFFF - torch.arange(c["vocab"], device="cuda"))
        index = 0xFFFFFFFF - (torch.topk(key, min(c["top"], c["vocab"]), dim=1).values & 0xFFFFFFFF)
        value = logp.gather(1, index).masked_fill(~kept[:, None], -math.inf)
        index = torch.where(value == -math.inf, -1, index).int()
        more = c["top"] - index.shape[1]
        o["top_logprob"] = torch.cat([value, value.new_full((c["rows"], more), -math.inf)], 1)
        o["top_index"] = torch.cat([index, index.new_full((c["rows"], more), -1)], 1)
    if c["step"] == "train":
        g, ge = s["g"].masked_fill(~kept, 0.0)[:, None], s["ge"].masked_fill(~kept, 0.0)[:, None]
        dz = -g * p - ge * (plogp + p * entropy)
        dz.scatter_add_(1, token, g)
        o["dlogits"] = (dz * c["scale"]).to(s["logits"].dtype)
    return o


def _plain_distill(s):
    c = s["case"]
    has = s["index"] >= 0
    index = s["index"].clamp(min=0)
    score = (s["teacher"].float() * c["scale"]).masked_fill(~has, -math.inf)
    if s["lse"] is not None:
        logq = score - s["lse"][:, None]
    else:
        top = score.amax(1, keepdim=True)
        score = score - torch.where(top == -math.inf, 0.0, top)
        total = torch.exp(score).sum(1, keepdim=True)
        logq = score - torch.log(torch.where(total == 0, 1.0, total))
    q = torch.exp(logq)
    t, log_sum = _plain_softmax(s)
    logp = t - log_sum
    loss = torch.where(q == 0, 0.0, q * (logq - logp.gather(1, index))).sum(1)
    dz = torch.exp(logp) * q.sum(1, keepdim=True)
    dz.scatter_add_(1, index, -q)
    return {"loss": loss, "dlogits": (dz * (s["g"] * c["scale"])[:, None]).to(s["logits"].dtype)}


# ---------------------------------------------------------------------------
# the package's entry points
# ---------------------------------------------------------------------------
def _own_norm(s, mfx):
    c = s["case"]
    args = dict(residual=s["residual"], eps=EPS, weight_offset=c["offset"])
    if c["quant"] != "none":
        q, scale, h, _ = mfx.mfx_add_rmsnorm_quant_fwd(
            s["x"], s["weight"], group=c["group"], q_dtype=DT[c["quant"]],
            scale_dtype=torch.float8_e8m0fnu if c["scales"] == "e8m0" else torch.float32, **args)
        o = {"q": q, "scale": scale}
        return o if h is None else {**o, "h": h}
    train = c["step"] == "train"
    y, h, rstd = mfx.mfx_add_rmsnorm_fwd(s["x"], s["weight"], need_rstd=train, **args)
    o = {"y": y} if h is None else {"y": y, "h": h}
    if train:
        o["dx"], dresidual, o["dweight"] = mfx.mfx_add_rmsnorm_bwd(
            s["dy"], s["x"] if h is None else h, rstd, s["weight"], dh=s["dh"], weight_offset=c["offset"],
            residual_dtype=None if h is None else h.dtype)
        if h is not None:
            o["dresidual"] = dresidual
    return o


def _own_logprobs(s, mfx):
    c = s["case"]
    train = c["step"] == "train"
    logprob, entropy, value, index, stats = mfx.mfx_token_logprobs_fwd(
        s["logits"], s["tokens"], scale=c["scale"], top=c["top"], need_stats=train)
    o = {"logprob": logprob, "entropy": entropy}
    if c["top"]:
        o["top_logprob"], o["top_index"] = value, index
    if train:
        o["dlogits"] = mfx.mfx_token_logprobs_bwd(s["g"], s["ge"], s["logits"], s["tokens"], stats, scale=c["scale"])
    return o


def _own_distill(s, mfx):
    c = s["case"]
    args = dict(scale=c["scale"], teacher_lse=s["lse"])
    data = (s["logits"], s["index"], s["teacher"])
    if c["step"] == "fused":
        loss, dlogits = mfx.mfx_topk_distill_fwd_bwd(*data, s["g"], **args)
    else:
        loss, stats = mfx.mfx_topk_distill_fwd(*data, **args)
        dlogits = mfx.mfx_topk_distill_bwd(s["g"], *data, stats, **args)
    return {"loss": loss, "dlogits": dlogits}


def run(s):
    op = s["case"]["op"]
    if own:
        import elementwise_epilogues_transformer_gb300 as mfx

        return {"norm": _own_norm, "logprobs": _own_logprobs, "distill": _own_distill}[op](s, mfx)
    return {"norm": _plain_norm, "logprobs": _plain_logprobs, "distill": _plain_distill}[op](s)


def work(c):
    """Bytes of the inputs and outputs, each once, and operations of one pass."""
    size = {"none": 0, "bf16": 2, "fp32": 4, "e4m3": 1, "e5m2": 1, "e8m0": 1}
    z = size[c["dtype"]]
    if c["op"] == "norm":
        n, r, w = c["rows"] * c["cols"], size[c["residual"]], c["cols"] * size[c["weight"]]
        each = z + 2 * r  # x, the residual before and after
        if c["quant"] != "none":
            groups = c["rows"] * (-(-c["cols"] // c["group"]) if c["group"] else 1)
            return {"bytes": n * (each + 1) + w + groups * size[c["scales"]], "flops": n * 7}
        if c["step"] == "infer":
            return {"bytes": n * (each + z) + w, "flops": n * 5}
        # y; dy, dh, dx, dresidual, and dweight
        return {"bytes": n * (each + 3 * z + 2 * r) + 2 * w, "flops": n * 16}
    n = c["rows"] * c["vocab"]
    if c["op"] == "logprobs":
        train = c["step"] == "train"
        lost = 1 - c["lost"]  # rows that are left out need not be read
        return {"bytes": int(n * z * (lost + train)) + c["rows"] * (16 + 8 * c["top"] + 8 * train),
                "flops": n * (12 if train else 6)}
    return {"bytes": 2 * n * z + c["rows"] * (c["k"] * (8 + size[c["teacher"]]) + 8), "flops": n * 8}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, apart from the above
# ---------------------------------------------------------------------------
def _exact_norm(c, s):
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
    w = s["weight"].double() + c["offset"]
    r = (h.square().sum(1) / c["cols"] + EPS).rsqrt()
    y = torch.einsum("rc,r,c->rc", h, r, w)
    o = {} if s["residual"] is None else {"h": h}
    if c["quant"] != "none":
        n, most = c["group"] or c["cols"], LARGEST[c["quant"]]
        scales = torch.stack([part.abs().max(1).values / most for part in y.split(n, 1)], 1)
        if c["scales"] == "e8m0":
            scales = torch.exp2(torch.ceil(torch.log2(scales.float().double().clamp(min=2.0 ** -126))))
        scales = torch.where(scales == 0, 1.0, scales)
        o["scale"] = scales
        o["q"] = y / scales.repeat_interleave(n, 1)[:, :c["cols"]]
        return o
    o["y"] = y
    if c["step"] == "train":
        kept = (s["x"] if s["residual"] is None else h.to(s["residual"].dtype)).double()
        dy = s["dy"].double()
        dot = torch.einsum("rc,c,rc->r", dy, w, kept)
        d = dy * w * r[:, None] - kept * (dot * r ** 3 / c["cols"])[:, None]
        if s["residual"] is not None:
            d += s["dh"].double()
            o["dresidual"] = d
        o["dx"] = d
        o["dweight"] = torch.einsum("rc,rc,r->c", dy, kept, r)
    return o


def _pieces(c):
    """Ranges of rows that 64 bits have room for."""
    step = max(1, (1 << 26) // c["vocab"])
    return [slice(i, min(i + step, c["rows"])) for i in range(0, c["rows"], step)]


def _exact_logprobs(c, s):
    rows, train = c["rows"], c["step"] == "train"
    o = {"logprob": torch.zeros(rows, dtype=torch.float64, device="cuda")}
    o["entropy"] = torch.zeros_like(o["logprob"])
    if c["top"]:
        o["top_logprob"] = torch.full((rows, c["top"]), -math.inf, dtype=torch.float64, device="cuda")
        o["top_index"] = None
    if train:
        o["dlogits"] = torch.zeros((rows, c["vocab"]), dtype=torch.float64, device="cuda")
    for at in _pieces(c):
        kept = torch.nonzero(s["tokens"][at] >= 0)[:, 0] + at.start
        z = s["logits"][kept].double() * c["scale"]
        token = s["tokens"][kept]
        logp = torch.log_softmax(z, 1)
        p = logp.exp()
        entropy = torch.special.entr(p).sum(1)
        every = torch.arange(kept.numel(), device="cuda")
        o["logprob"][kept], o["entropy"][kept] = logp[every, token], entropy
        if c["top"]:
            best = torch.sort(logp, 1, descending=True).values[:, :c["top"]]
            o["top_logprob"][kept, :best.shape[1]] = best
        if train:
            g, ge = s["g"][kept].double(), s["ge"][kept].double()
            d = torch.special.entr(p) * ge[:, None] - p * (g + ge * entropy)[:, None]
            d[every, token] += g
            o["dlogits"][kept] = d * c["scale"]
    return o


def _exact_distill(c, s):
    loss = torch.zeros(c["rows"], dtype=torch.float64, device="cuda")
    dlogits = torch.zeros((c["rows"], c["vocab"]), dtype=torch.float64, device="cuda")
    for at in _pieces(c):
        logp = torch.log_softmax(s["logits"][at].double() * c["scale"], 1)
        index, t = s["index"][at], s["teacher"][at].double() * c["scale"]
        t = torch.where(index < 0, -math.inf, t)
        lse = torch.logsumexp(t, 1) if s["lse"] is None else s["lse"][at].double()
        logq = t - torch.where(lse == -math.inf, 0.0, lse)[:, None]
        q = logq.exp()
        loss[at] = -(torch.special.entr(q) + q * logp.gather(1, index.clamp(min=0))).sum(1)
        d = logp.exp() * q.sum(1, keepdim=True)
        d.scatter_add_(1, index.clamp(min=0), -q)
        dlogits[at] = d * s["g"][at].double()[:, None] * c["scale"]
    return {"loss": loss, "dlogits": dlogits}


def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "logprobs": _exact_logprobs, "distill": _exact_distill}[c["op"]](c, s)
