"""Measured cases of three operators around a transformer layer: the softmax of
attention scores with a learned relative position bias and dropout, dropout
whose mask is never stored, and tokens sorted by expert and back.

``run`` computes them in their plain form (elementary torch operations in
32 bits, 64 where sums are long), or through the package's entry points where
``own`` is true.  ``exact`` is the same from the definitions in 64 bits.

Definitions:

* scores: s[b,h,q,k] = x * scale + table[bucket(k - pos_q), h] + mask, with
  pos_q = q_start + seq_start[b] + q; causal calls leave out k > pos_q.
  P = softmax over k (a row with nothing left is zero);
  y = keep * P / (1 - p).  Backward from dy: dP = keep * dy / (1 - p),
  dS = P * (dP - sum_k dP P), dx = scale * dS, and dtable sums dS over the
  positions of each bucket.
* buckets: distances n below half the buckets of a direction have one each;
  the others grow geometrically up to max_distance, the last one open.
* dropout: element e keeps its value where 16-bit word e % 8 of the
  Philox4x32-10 block e // 8 (key: seed, counter: block and offset) is at
  least ceil(65536 p), and is then scaled by 1 / (1 - p).
* sorting: slots (token, choice) are laid out by expert, by slot index within
  one; each expert's rows start at a multiple of `align`; slots without an
  expert, or past an expert's capacity, have no row.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _scores(name, b, np, sq, sk, dtype, step, p=0.0, mask="none", causal=False, bidirectional=True, buckets=32,
            max_distance=128, table="bf16", ragged=False, elem_base=0):
    c = dict(op="scores", b=b, np=np, sq=sq, sk=sk, dtype=dtype, step=step, p=p, mask=mask, causal=causal,
             bidirectional=bidirectional, buckets=buckets, max_distance=max_distance, table=table, ragged=ragged,
             elem_base=elem_base)
    return dict(c, name=name) if name else c


def _dropout(name, form, rows, cols, dtype, residual, p, elem_base=0):
    c = dict(op="dropout", form=form, rows=rows, cols=cols, dtype=dtype, residual=residual, p=p, elem_base=elem_base)
    return dict(c, name=name) if name else c


def _experts(name, tokens, cols, experts, topk, dtype, step, weights="out", align=1, capacity=0, lost=0.0):
    c = dict(op="experts", tokens=tokens, cols=cols, experts=experts, topk=topk, dtype=dtype, step=step,
             weights=weights, align=align, capacity=capacity, lost=lost)
    return dict(c, name=name) if name else c


def listed():
    return [
        # an encoder's attention scores at the softmax benchmark's size, forward and backward
        _scores("scores train 2x32x4096x4096", 2, 32, 4096, 4096, "bf16", "train", p=0.1),
        # a decoder's causal scores with a padding mask and one-directional buckets
        _scores("scores causal pad 4x12x1024", 4, 12, 1024, 1024, "bf16", "train", p=0.1, mask="pad", causal=True,
                bidirectional=False),
        # cross-shaped scores of odd sizes in fp32, a full additive mask, no dropout
        _scores("scores odd fp32 3x7x333x1001", 3, 7, 333, 1001, "fp32", "train", mask="full", table="fp32"),
        # one new token for each of many sequences of different lengths over a long cache
        _scores("scores decode 32x32x8192", 32, 32, 1, 8192, "bf16", "decode", causal=True, bidirectional=False,
                ragged=True),
        # one new token of one sequence over a very long cache: few rows, long ones
        _scores("scores decode 1x16x131072", 1, 16, 1, 131072, "bf16", "decode", bidirectional=False),
        # one new token early in one short sequence: latency
        _scores("scores decode 1x8x77", 1, 8, 1, 77, "bf16", "decode", bidirectional=False),
        # the residual path of a layer, forward and backward, fp32 residual stream
        _dropout("residual 16384x4096", "residual", 16384, 4096, "bf16", "fp32", 0.1),
        # dropout of embeddings at an odd width, forward and backward
        _dropout("embedding 32768x4099", "plain", 32768, 4099, "bf16", "bf16", 0.1),
        # the residual path of a small fp32 model
        _dropout("residual fp32 512x1024", "residual", 512, 1024, "fp32", "fp32", 0.5),
        # few large experts, two per token, forward and backward
        _experts("experts train 16384x4096 2/8", 16384, 4096, 8, 2, "bf16", "train"),
        # many small experts with aligned rows and a capacity; the weight goes through the activation
        _experts("experts train 8192x2048 8/128", 8192, 2048, 128, 8, "bf16", "train", weights="act", align=16,
                 capacity=640, lost=0.02),
        # the same routing for a decode batch
        _experts("experts decode 16x4096 8/64", 16, 4096, 64, 8, "bf16", "decode"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    return v + 1 if v == 3072 else v


def draw(rng: random.Random):
    kind = rng.choice(["scores", "scores", "decode", "dropout", "experts", "experts"])
    if kind == "scores":
        b, np = rng.randint(1, 4), rng.choice([1, 4, 6, 12, 16, 32])
        sq = _log(rng, 1, 4096)
        sk = sq if rng.random() < 0.4 else _log(rng, 1, 16384)
        while b * np * sq * sk > 1 << 28:
            sq, sk = max(1, sq * 3 // 4), max(1, sk * 3 // 4)
            sq, sk = sq + (sq == 3072), sk + (sk == 3072)
        bid = rng.random() < 0.5
        return _scores(None, b, np, sq, sk, rng.choice(["bf16", "bf16", "fp32"]), "train",
                       p=rng.choice([0.0, 0.1, 0.25]), mask=rng.choice(["none", "pad", "full", "lowest"]),
                       causal=not bid and rng.random() < 0.7, bidirectional=bid, buckets=rng.choice([8, 32, 64]),
                       max_distance=rng.choice([64, 128, 800]), table=rng.choice(["bf16", "fp32"]),
                       ragged=rng.random() < 0.3, elem_base=rng.choice([0, 0, 8 * rng.randint(1, 1 << 33)]))
    if kind == "decode":
        b, np = _log(rng, 1, 64), rng.choice([4, 8, 12, 32])
        return _scores(None, b, np, 1, _log(rng, 1, 131072 if b * np <= 512 else 16384),
                       rng.choice(["bf16", "bf16", "fp32"]), "decode", mask=rng.choice(["none", "none", "pad"]),
                       causal=rng.random() < 0.7, bidirectional=False, buckets=rng.choice([16, 32]),
                       max_distance=rng.choice([128, 512]), table=rng.choice(["bf16", "fp32"]),
                       ragged=rng.random() < 0.7)
    if kind == "dropout":
        form = rng.choice(["residual", "plain"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return _dropout(None, form, _log(rng, 1, 32768), rng.choice([1024, 4096, 4099, _log(rng, 1, 8192)]), dtype,
                        dtype if form == "plain" else rng.choice(["bf16", "fp32"]), rng.choice([0.1, 0.25, 0.5]),
                        elem_base=rng.choice([0, 0, rng.randint(1, 1 << 35)]))
    experts = rng.choice([4, 8, 60, 64, 128, 256])
    topk = rng.choice([1, 2, 4, 8]) if experts >= 8 else rng.choice([1, 2])
    cols = rng.choice([1024, 2048, 4096, _log(rng, 64, 8192)])
    tokens = max(1, min(_log(rng, 1, 32768), (1 << 27) // (cols * topk)))
    step = "decode" if tokens <= 64 else "train"
    return _experts(None, tokens, cols, experts, topk, rng.choice(["bf16", "bf16", "fp32"]), step,
                    weights=rng.choice(["out", "act"]), align=rng.choice([1, 1, 16, 128]) if step == "train" else 1,
                    capacity=rng.choice([0, max(1, tokens * topk * 5 // (experts * 4))]),
                    lost=rng.choice([0.0, 0.05]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _rows(c):
    """Rows that the sorted layout needs at most."""
    slots = c["tokens"] * c["topk"]
    return slots + min(c["experts"], slots) * (c["align"] - 1)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "seed": 1234 + seed, "offset": 7 * seed}
    if c["op"] == "scores":
        b, np, sq, sk, dt = c["b"], c["np"], c["sq"], c["sk"], DT[c["dtype"]]
        # scores of unit-variance vectors of 64 elements
        s["scale"] = 0.125
        s["x"] = _normal(g, (b, np, sq, sk), dt, 8.0)
        s["dy"] = _normal(g, (b, np, sq, sk), dt) if c["step"] == "train" else None
        s["table"] = _normal(g, (c["buckets"], np), DT[c["table"]])
        lengths = torch.randint((sk + 1) // 2, sk + 1, (b,), generator=g, device="cuda")
        if c["mask"] == "pad":
            s["mask"] = torch.where(torch.arange(sk, device="cuda") < lengths[:, None], 0.0, -math.inf)
            s["mask"] = s["mask"].to(dt).reshape(b, 1, 1, sk)
        elif c["mask"] == "full":
            s["mask"] = _normal(g, (1, 1, sq, sk), dt)
            s["mask"][torch.rand((1, 1, sq, sk), generator=g, device="cuda") < 0.1] = -math.inf
        elif c["mask"] == "lowest":  # padding by the type's lowest value; the first query sees nothing else
            s["mask"] = torch.where(torch.arange(sk, device="cuda") < lengths[:, None], 0.0, torch.finfo(dt).min)
            s["mask"] = s["mask"].to(dt).reshape(b, 1, 1, sk).expand(b, 1, sq, sk).contiguous()
            s["mask"][:, :, 0] = torch.finfo(dt).min
        else:
            s["mask"] = None
        # positions: ragged calls have sequences of different lengths, others end at the last key
        s["q_start"] = 0 if c["ragged"] else max(0, sk - sq) if c["step"] == "train" else sk - 1
        s["seq_start"] = (lengths - 1).to(torch.int32) if c["ragged"] else None
    elif c["op"] == "dropout":
        shape, dt = (c["rows"], c["cols"]), DT[c["dtype"]]
        s["x"], s["g"] = _normal(g, shape, dt), _normal(g, shape, dt)
        s["bias"] = _normal(g, (c["cols"],), dt, 0.02)
        s["residual"] = _normal(g, shape, DT[c["residual"]]) if c["form"] == "residual" else None
    else:
        t, k, e, h, dt = c["tokens"], c["topk"], c["experts"], c["cols"], DT[c["dtype"]]
        # a router's choices: distinct experts by score, some experts liked more than others
        logits = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn((e,), generator=g, device="cuda")
        top, choice = torch.topk(logits, k, dim=1)
        s["weight"] = torch.exp(top - top.amax(1, keepdim=True))
        s["weight"] = s["weight"] / s["weight"].sum(1, keepdim=True)
        s["expert_of"] = torch.where(torch.rand((t, k), generator=g, device="cuda") < c["lost"], -1, choice)
        s["expert_of"] = s["expert_of"].to(torch.int32)
        s["x"], s["y"] = _normal(g, (t, h), dt), _normal(g, (_rows(c), h), dt)
        if c["step"] == "train":
            s["g"], s["gp"] = _normal(g, (t, h), dt), _normal(g, (_rows(c), h), dt)
            s["gw"] = _normal(g, (_rows(c),), torch.float32) if c["weights"] == "act" else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _thresholds(c):
    """Smallest distance of each bucket of one direction, in whole numbers: the first half is 0, 1, 2, ..., and
    bucket first + j begins at the least n with (n / first)^steps >= (max_distance / first)^j."""
    n = c["buckets"] // 2 if c["bidirectional"] else c["buckets"]
    first = n // 2
    steps, far = n - first, c["max_distance"]
    return list(range(1, first + 1)) + [next(
        d for d in range(max(first, int(first * (far / first) ** (j / steps)) - 2), far + 1)
        if d ** steps * first ** j >= far ** j * first ** steps) for j in range(1, steps)]


def _buckets(c, rel):
    """Bucket of each relative position (key minus query)."""
    n = rel.abs() if c["bidirectional"] else (-rel).clamp(min=0)
    below = torch.tensor(_thresholds(c), device=rel.device)
    bucket = torch.bucketize(n, below, right=True)
    return bucket + (rel > 0) * (c["buckets"] // 2) if c["bidirectional"] else bucket


def _positions(s):
    c = s["case"]
    start = s["q_start"] + (s["seq_start"].long() if s["seq_start"] is not None else
                            torch.zeros(1, dtype=torch.long, device="cuda"))
    pos = start[:, None] + torch.arange(c["sq"], device="cuda")
    return torch.arange(c["sk"], device="cuda") - pos[..., None]  # [b or 1, sq, sk]


def _keep(n, base, p, seed, offset):
    """Which of the elements base .. base + n - 1 are kept."""
    first = base // 8
    count = (base + n - 1) // 8 - first + 1
    low = 0xFFFFFFFF
    block = torch.arange(first, first + count, device="cuda")
    c0, c1 = block & low, block >> 32
    c2, c3 = torch.full_like(block, offset & low), torch.full_like(block, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products; the sign bit is only a bit
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], 1).to(torch.int32).view(torch.int16).reshape(-1).to(torch.int32) & 0xFFFF
    return words[base - 8 * first:base - 8 * first + n] >= min(65535, math.ceil(p * 65536))


def _plain_scores(s):
    c = s["case"]
    b, np, sq, sk = s["x"].shape
    x = s["x"].float()
    rel = _positions(s)
    bucket = _buckets(c, rel)
    scores = x * s["scale"] + s["table"].float()[bucket].permute(0, 3, 1, 2)
    left_out = (rel > 0)[:, None] if c["causal"] else torch.zeros((1, 1, 1, 1), dtype=torch.bool, device="cuda")
    if s["mask"] is not None:
        mask = s["mask"].float().masked_fill(left_out, -math.inf)
        # a softmax does not change when its row is shifted: rows of lowest values keep their scores so
        shift = mask.amax(-1, keepdim=True)
        left_out = mask == -math.inf
        scores = scores + (mask - torch.where(shift == -math.inf, 0.0, shift))
    scores = scores.masked_fill(left_out, -math.inf)
    top = scores.amax(-1, keepdim=True)
    P = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = P.sum(-1, keepdim=True)
    P = P / torch.where(total == 0, 1.0, total)
    scale = 1.0 / (1.0 - c["p"])
    keep = _keep(P.numel(), c["elem_base"], c["p"], s["seed"], s["offset"]).view(P.shape) if c["p"] else None
    y = (P * scale).masked_fill(~keep, 0.0).to(s["x"].dtype) if c["p"] else P.to(s["x"].dtype)
    if c["step"] != "train":
        return {"y": y}
    dP = (s["dy"].float() * scale).masked_fill(~keep, 0.0) if c["p"] else s["dy"].float()
    dS = P * (dP - (dP * P).sum(-1, keepdim=True))
    one = (bucket[..., None] == torch.arange(c["buckets"], device="cuda")).double()  # long sums: 64 bits
    if bucket.shape[0] == 1:
        dtable = one.view(sq * sk, -1).t() @ dS.sum(0, dtype=torch.float64).view(np, sq * sk).t()
    else:
        dtable = (one.view(b, sq * sk, -1).transpose(1, 2) @ dS.double().view(b, np, sq * sk).transpose(1, 2)).sum(0)
    return {"y": y, "dx": (dS * s["scale"]).to(s["x"].dtype), "dtable": dtable.to(s["table"].dtype)}


def _plain_dropout(s):
    c = s["case"]
    keep = _keep(s["x"].numel(), c["elem_base"], c["p"], s["seed"], s["offset"]).view(s["x"].shape)
    scale, dt = 1.0 / (1.0 - c["p"]), s["x"].dtype
    dx = (s["g"].float() * scale).masked_fill(~keep, 0.0).to(dt)
    if c["form"] == "plain":
        return {"out": (s["x"].float() * scale).masked_fill(~keep, 0.0).to(dt), "dx": dx}
    v = ((s["x"].float() + s["bias"].float()) * scale).masked_fill(~keep, 0.0) + s["residual"].to(dt).float()
    return {"out": v.to(dt), "dx": dx, "dresidual": s["g"].to(s["residual"].dtype)}


def _plain_sort(s):
    c = s["case"]
    e, slots = c["experts"], c["tokens"] * c["topk"]
    key = s["expert_of"].view(-1).long()
    key = torch.where((key < 0) | (key >= e), e, key)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(e + 1, dtype=torch.long, device="cuda").index_add_(0, key, torch.ones_like(key))
    rank = torch.empty_like(key)
    begin = torch.cumsum(counts, 0) - counts
    rank[order] = torch.arange(slots, device="cuda") - begin[key[order]]
    kept = counts[:e].clamp(max=c["capacity"]) if c["capacity"] else counts[:e]
    offsets = torch.zeros(e + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum((kept + c["align"] - 1) // c["align"] * c["align"], 0)
    has = (key < e) & (rank < (c["capacity"] or slots))
    row_of = torch.where(has, offsets[key.clamp(max=e - 1)] + rank, -1)
    slot_of = torch.full((_rows(c) + 1,), -1, dtype=torch.long, device="cuda")  # the last: slots without a row
    slot_of[row_of] = torch.where(has, torch.arange(slots, device="cuda"), -1)
    return row_of.view(c["tokens"], -1), slot_of[:-1], offsets, kept


def _plain_experts(s):
    c = s["case"]
    row_of, slot_of, offsets, kept = _plain_sort(s)
    dt, act = s["x"].dtype, c["weights"] == "act"
    filled, has = (slot_of >= 0), (row_of >= 0)[..., None]
    token = slot_of.clamp(min=0) // c["topk"]
    out = {"row_of": row_of.int(), "slot_of": slot_of.int(), "offsets": offsets.int(), "counts": kept.int()}
    out["xp"] = s["x"][token].masked_fill(~filled[:, None], 0.0)
    w = s["weight"][..., None]
    if act:
        out["wp"] = s["weight"].view(-1)[slot_of.clamp(min=0)].masked_fill(~filled, 0.0)
    y = s["y"].float()[row_of.clamp(min=0)].masked_fill(~has, 0.0)
    out["out"] = (y if act else y * w).sum(1).to(dt)
    if c["step"] == "train":
        dy = s["g"].float()[token]
        dy = dy if act else dy * s["weight"].view(-1)[slot_of.clamp(min=0)][:, None]
        out["dy"] = dy.masked_fill(~filled[:, None], 0.0).to(dt)
        out["dx"] = s["gp"].float()[row_of.clamp(min=0)].masked_fill(~has, 0.0).sum(1).to(dt)
        out["dw"] = (s["gw"][row_of.clamp(min=0)].masked_fill(~has[..., 0], 0.0) if act
                     else (s["g"].float()[:, None] * y).sum(-1, dtype=torch.float64).float())
    return out


# ---------------------------------------------------------------------------
# the package's entry points
# ---------------------------------------------------------------------------
def _own_scores(s, mfx):
    c = s["case"]
    args = dict(table=s["table"], mask=s["mask"], max_distance=c["max_distance"], bidirectional=c["bidirectional"],
                causal=c["causal"], q_start=s["q_start"], seq_start=s["seq_start"], p=c["p"], seed=s["seed"],
                offset=s["offset"], elem_base=c["elem_base"])
    if c["step"] != "train":
        return {"y": mfx.mfx_relbias_softmax_dropout_fwd(s["x"], s["scale"], need_stats=False, **args)[0]}
    y, stats = mfx.mfx_relbias_softmax_dropout_fwd(s["x"], s["scale"], **args)
    dx, dtable = mfx.mfx_relbias_softmax_dropout_bwd(s["dy"], s["x"], stats, s["scale"], **args)
    return {"y": y, "dx": dx, "dtable": dtable}


def _own_dropout(s, mfx):
    c = s["case"]
    key = (c["p"], s["seed"], s["offset"], c["elem_base"])
    if c["form"] == "plain":
        return {"out": mfx.mfx_dropout_fwd(s["x"], *key), "dx": mfx.mfx_dropout_bwd(s["g"], *key)}
    out = mfx.mfx_bias_dropout_add_train_nomask(s["x"], s["bias"], s["residual"], *key)
    dx, dresidual = mfx.mfx_bias_dropout_add_bwd(s["g"], None, *key, residual_dtype=s["residual"].dtype)
    return {"out": out, "dx": dx, "dresidual": dresidual}


def _own_experts(s, mfx):
    c = s["case"]
    act = c["weights"] == "act"
    row_of, slot_of, offsets, counts = mfx.mfx_moe_sort(s["expert_of"], c["experts"], align=c["align"],
                                                        capacity=c["capacity"])
    xp, wp = mfx.mfx_moe_permute_fwd(s["x"], row_of, slot_of, weight=s["weight"] if act else None)
    o = {"row_of": row_of, "slot_of": slot_of, "offsets": offsets, "counts": counts, "xp": xp}
    if act:
        o["wp"] = wp
    w = None if act else s["weight"]
    o["out"] = mfx.mfx_moe_unpermute_fwd(s["y"], row_of, weight=w)
    if c["step"] == "train":
        o["dy"], dw = mfx.mfx_moe_unpermute_bwd(s["g"], s["y"], row_of, slot_of, weight=w)
        o["dx"], dwp = mfx.mfx_moe_permute_bwd(s["gp"], row_of, g_weight=s["gw"])
        o["dw"] = dwp if act else dw
    return o


def run(s):
    op = s["case"]["op"]
    if own:
        import elementwise_epilogues_transformer_gb300 as mfx

        return {"scores": _own_scores, "dropout": _own_dropout, "experts": _own_experts}[op](s, mfx)
    return {"scores": _plain_scores, "dropout": _plain_dropout, "experts": _plain_experts}[op](s)


def work(c):
    """Bytes of the inputs and outputs, each once, and operations of one pass."""
    size = {"bf16": 2, "fp32": 4}
    z = size[c["dtype"]]
    if c["op"] == "scores":
        n = c["b"] * c["np"] * c["sq"] * c["sk"]
        train = c["step"] == "train"
        # inputs that a causal call does not look at need not be read (whole rows of keys at or before the query)
        seen = n
        if c["causal"] and not c["ragged"] and train:
            start = max(0, c["sk"] - c["sq"])
            seen = c["b"] * c["np"] * sum(min(c["sk"], start + q + 1) for q in range(c["sq"]))
        elif c["causal"] and c["ragged"]:
            seen = n * 3 // 4  # lengths are uniform between half and all of the keys
        mask = {"none": 0, "pad": c["b"] * c["sk"], "full": c["sq"] * c["sk"], "lowest": c["b"] * c["sq"] * c["sk"]}
        moved = seen * (2 if train else 1) + n * (2 if train else 1) + mask[c["mask"]]
        return {"bytes": moved * z + c["buckets"] * c["np"] * size[c["table"]], "flops": n * (16 if train else 6)}
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        more = 2 * size[c["residual"]] if c["form"] == "residual" else 0
        return {"bytes": n * (4 * z + more), "flops": n * 4}
    t, r, h = c["tokens"], c["tokens"] * c["topk"], c["cols"]
    maps = 4 * (3 * r + 2 * c["experts"])
    elements = (t + r) + (r + t)  # tokens to rows, and rows to tokens
    if c["step"] == "train":
        elements += (t + r) + (r + t)
    return {"bytes": elements * h * z + maps, "flops": 2 * r * h * (3 if c["step"] == "train" else 1)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, apart from the above
# ---------------------------------------------------------------------------
def _exact_keep(n, base, p, seed, offset):
    """The same generator with its products formed from 16-bit halves."""
    first, last = base // 8, (base + n - 1) // 8

    def wide(a, m):  # (low, high) 32 bits of a * m
        ah, al, mh, ml = a >> 16, a & 0xFFFF, m >> 16, m & 0xFFFF
        mid = ah * ml + ((al * ml) >> 16)
        mid2 = al * mh + (mid & 0xFFFF)
        return ((mid2 & 0xFFFF) << 16) | ((al * ml) & 0xFFFF), ah * mh + (mid >> 16) + (mid2 >> 16)

    ctr = torch.arange(first, last + 1, dtype=torch.int64, device="cuda")
    v = [ctr % 2**32, ctr // 2**32, torch.zeros_like(ctr) + offset % 2**32, torch.zeros_like(ctr) + offset // 2**32]
    key = [seed % 2**32, seed // 2**32]
    for i in range(10):
        l0, h0 = wide(v[0], 0xD2511F53)
        l1, h1 = wide(v[2], 0xCD9E8D57)
        v = [h1 ^ v[1] ^ ((key[0] + i * 0x9E3779B9) % 2**32), l1, h0 ^ v[3] ^ ((key[1] + i * 0xBB67AE85) % 2**32), l0]
    limit = min(65535, math.ceil(p * 65536))
    kept = torch.empty((last + 1 - first, 8), dtype=torch.bool, device="cuda")
    for j in range(4):
        kept[:, 2 * j] = v[j] % 65536 >= limit
        kept[:, 2 * j + 1] = v[j] // 65536 >= limit
    return kept.view(-1)[base % 8:base % 8 + n]


def _exact_bucket(c, rel):
    half = c["buckets"] // 2 if c["bidirectional"] else c["buckets"]
    n = (rel.abs() if c["bidirectional"] else torch.clamp(-rel, min=0)).double()
    first = half // 2
    # the smallest addend lifts whole powers over their border; others are further from it than that
    far = first + torch.floor(torch.log(torch.clamp(n, min=1) / first) / math.log(c["max_distance"] / first)
                              * (half - first) + 1e-9)
    bucket = torch.where(n < first, n, torch.clamp(far, max=half - 1)).long()
    return torch.where(rel > 0, bucket + half, bucket) if c["bidirectional"] else bucket


def _exact_scores(c, s):
    b, np, sq, sk = s["x"].shape
    n, train = np * sq * sk, c["step"] == "train"
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    dx = torch.empty_like(y) if train else None
    dtable = torch.zeros(c["buckets"], np, dtype=torch.float64, device="cuda")
    k = torch.arange(sk, device="cuda")
    by = np if n <= 1 << 26 else 1  # heads at a time
    for i in range(b):
        q = s["q_start"] + torch.arange(sq, device="cuda")
        if s["seq_start"] is not None:
            q = q + int(s["seq_start"][i])
        rel = k[None, :] - q[:, None]
        bucket = _exact_bucket(c, rel)
        if train:
            flat = bucket.view(-1)
        for h in range(0, np, by):
            at = slice(h, h + by)
            t = s["x"][i, at].double() * s["scale"] + s["table"][:, at].double().t()[:, bucket]
            if s["mask"] is not None:
                m = s["mask"][i if s["mask"].shape[0] > 1 else 0].double()
                if c["causal"]:
                    m = torch.where(rel > 0, -math.inf, m)
                high = m.max(-1, keepdim=True).values
                t = t + torch.where(m == -math.inf, -math.inf, m - torch.where(high == -math.inf, 0.0, high))
            elif c["causal"]:
                t = torch.where(rel > 0, -math.inf, t)
            lse = torch.logsumexp(t, -1, keepdim=True)
            P = torch.where(lse == -math.inf, 0.0, torch.exp(t - torch.where(lse == -math.inf, 0.0, lse)))
            del t
            kept = None
            if c["p"]:
                kept = _exact_keep(P.numel(), c["elem_base"] + (i * np + h) * sq * sk, c["p"], s["seed"], s["offset"])
                kept = kept.view(P.shape).double() / (1.0 - c["p"])
            y[i, at] = P if kept is None else P * kept
            if train:
                d = s["dy"][i, at].double()
                d = d if kept is None else d * kept
                d = P * (d - (d * P).sum(-1, keepdim=True))
                dx[i, at] = d * s["scale"]
                for j in range(d.shape[0]):
                    dtable[:, h + j] += torch.bincount(flat, weights=d[j].reshape(-1), minlength=c["buckets"])
    return {"y": y, "dx": dx, "dtable": dtable} if train else {"y": y}


def _exact_dropout(c, s):
    kept = _exact_keep(s["x"].numel(), c["elem_base"], c["p"], s["seed"], s["offset"]).view(s["x"].shape).double()
    kept = kept / (1.0 - c["p"])
    if c["form"] == "plain":
        return {"out": s["x"].double() * kept, "dx": s["g"].double() * kept}
    return {"out": (s["x"].double() + s["bias"].double()) * kept + s["residual"].to(s["x"].dtype).double(),
            "dx": s["g"].double() * kept, "dresidual": s["g"].double()}


def _exact_experts(c, s):
    t, k, e = c["tokens"], c["topk"], c["experts"]
    picks = s["expert_of"].cpu().numpy().reshape(-1)
    rows, at, first = [-1] * (t * k), 0, [[] for _ in range(e)]
    for slot, x in enumerate(picks.tolist()):
        if 0 <= x < e and (not c["capacity"] or len(first[x]) < c["capacity"]):
            first[x].append(slot)
    owner = [-1] * _rows(c)
    for mine in first:
        for r, slot in enumerate(mine):
            rows[slot], owner[at + r] = at + r, slot
        at += -(-len(mine) // c["align"]) * c["align"]
    rows = torch.tensor(rows, device="cuda").view(t, k)
    owner = torch.tensor(owner, device="cuda")
    act, train = c["weights"] == "act", c["step"] == "train"
    weight = s["weight"].double()
    real = owner >= 0
    xp = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    xp[real] = s["x"].double()[owner[real] // k]
    o = {"row_of": None, "slot_of": None, "offsets": None, "counts": None, "xp": xp}
    if act:
        o["wp"] = torch.zeros(owner.shape, dtype=torch.float64, device="cuda")
        o["wp"][real] = weight.view(-1)[owner[real]]
    o["out"] = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    if train:
        o["dx"], o["dy"] = torch.zeros_like(o["out"]), torch.zeros_like(xp)
        o["dw"] = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        on = rows[:, j] >= 0
        r, w = rows[on, j], 1.0 if act else weight[on, j][:, None]
        y = s["y"][r].double()
        o["out"][on] += y * w
        if train:
            g = s["g"][on].double()
            o["dx"][on] += s["gp"][r].double()
            o["dy"][r] = g * w
            o["dw"][on, j] = s["gw"][r].double() if act else (g * y).sum(-1)
    return o


def exact(c, seed):
    s = prepare(c, seed)
    return {"scores": _exact_scores, "dropout": _exact_dropout, "experts": _exact_experts}[c["op"]](c, s)
