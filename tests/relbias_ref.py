"""Plain 64-bit form of the relative-position-bias softmax with dropout, and
how far the kernels' fp32 arithmetic may be from it.

With u = 2^-24 (half a step of fp32, relative) and, per row, A the largest
|x * scale + bias| + |mask - its maximum| among the finite ones:
  a score is off by at most 3 u A (product-sum, mask difference, sum); its
  exponential by that, the rounding of the exponent (<= 4 u A: |s - m| <= 2A,
  formed with one product or difference and one addition) and the exponential
  itself (2 ulp, 4 u): u (7A + 4) relative.  The parts of a row are joined
  with one more exponential of an argument <= 2A, u (2A + 4), and summed with
  at most 128 additions in a row; numerator and denominator have all of these:
  P is off by at most rP = u (18A + 160) relative.  The backward forms P from
  the stored maximum and reciprocal sum, within the same; it is given
  rP = u (20A + 200).
"""
import math

import torch

import oracle as O

U = 2.0 ** -24
TINY = 2.0 ** -120  # results below are flushed


def thresholds(side, far):
    """First distance of the buckets first + 1 .. side - 1 in whole numbers."""
    first = side // 2
    steps = side - first
    out, n = [], first
    for j in range(1, steps):
        while n ** steps * first ** j < far ** j * first ** steps:
            n += 1
        out.append(n)
    return first, out


def bucket(rel, num, far, two):
    side = num // 2 if two else num
    first, borders = thresholds(side, far)
    n = rel.abs() if two else (-rel).clamp(min=0)
    u = n.clamp(max=first)
    for t in borders:
        u = u + (n >= t)
    return torch.where(rel > 0, u + side, u) if two else u


def keep_flags(shape, p, seed, offset, base):
    """The oracle's keep flags of a tensor."""
    n = math.prod(shape)
    z = torch.zeros(1, n).numpy()
    _, m = O.bias_dropout_add_train(z, z, None, p=p, seed=seed, offset=offset, elem_base=base)
    return torch.from_numpy(m.reshape(shape)).bool()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def reference(x, scale, table=None, mask=None, max_distance=128, bidirectional=True, causal=False, q_start=0,
              seq_start=None, p=0.0, seed=0, offset=0, elem_base=0, dy=None):
    """(y, tol_y) or, with dy, also (dx, tol_dx, dtable, tol_dtable); all float64 on x's device.  The tolerances
    hold for outputs of x's and table's dtype."""
    dev = x.device
    b, np_, sq, sk = x.shape
    pos = q_start + torch.arange(sq, device=dev)[None, :] + (
        seq_start.long()[:, None] if seq_start is not None else torch.zeros(b, 1, dtype=torch.long, device=dev))
    rel = torch.arange(sk, device=dev) - pos[..., None]  # [b, sq, sk]
    s = x.double() * scale
    if table is not None:
        bk = bucket(rel, table.shape[0], max_distance, bidirectional)
        s = s + table.double()[bk].permute(0, 3, 1, 2)
    size = s.abs()
    out = torch.zeros(b, np_, sq, sk, dtype=torch.bool, device=dev)
    if causal:
        out |= (rel > 0)[:, None]
    if mask is not None:
        m = mask.double().expand(b, np_, sq, sk).masked_fill(out, -math.inf)
        out = out | (m == -math.inf)
        top = m.amax(-1, keepdim=True)
        shifted = m - torch.where(top == -math.inf, 0.0, top)
        s = s + shifted
        near = shifted > -1e4  # the others weigh nothing
        size = torch.where(near, size + shifted.abs(), 0.0)
    s = s.masked_fill(out, -math.inf)
    size = size.masked_fill(out, 0.0)
    A = torch.nan_to_num(size, nan=0.0, posinf=0.0).amax(-1, keepdim=True)
    lse = torch.logsumexp(s, -1, keepdim=True)
    P = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse))
    P = P.masked_fill(out & ~torch.isnan(lse), 0.0)
    f = 1.0
    if p:
        f = keep_flags(x.shape, p, seed, offset, elem_base).to(dev).double() / (1.0 - torch.tensor(p).double().item())
    y = P * f
    tol_y = y.abs() * (U * (18 * A + 164) + half_step(x.dtype)) + TINY
    if dy is None:
        return y, tol_y
    dP = torch.where(P == 0, 0.0, dy.double() * f)
    D = (dP * P).sum(-1, keepdim=True)
    dS = P * (dP - D)
    rP = U * (20 * A + 200)
    errD = (rP + 132 * U) * (dP * P).abs().sum(-1, keepdim=True)
    err = P * ((dP - D).abs() * (rP + 2 * U) + 3 * U * dP.abs() + errD + U * D.abs()) + TINY
    dx = dS * scale
    tol_dx = abs(scale) * err + (half_step(x.dtype) + U) * (dx.abs() + abs(scale) * err) + TINY
    if table is None:
        return y, tol_y, dx, tol_dx, None, None
    # a slot or far sum takes at most 256 additions at these sizes, the block sums less
    num = table.shape[0]
    dt = torch.zeros(num, np_, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(dt)
    for u in range(num):
        at = (bk == u)[:, None]
        dt[u] = torch.where(at, dS, 0.0).sum((0, 2, 3))
        tol[u] = torch.where(at, err + 256 * U * dS.abs(), 0.0).sum((0, 2, 3))
    return y, tol_y, dx, tol_dx, dt, tol + half_step(table.dtype) * (dt.abs() + tol) + TINY


def close(got, want, tol, what):
    """Element by element; NaN where NaN is wanted."""
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    bad = ~nan & ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i}: {got[i].item():.9g}, "
                             f"want {want[i].item():.9g} +- {tol[i].item():.3g}")
