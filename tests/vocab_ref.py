"""64-bit forms of the norm, the token log probabilities and the distillation,
and how far 32-bit kernels may be from them.

A value stored in a type is off by at most half a step of it
(finfo.eps / 2 of the value); a 32-bit operation by U = 2^-24 of its result;
a sum of n terms formed by s sequential additions and a tree by at most
(s + tree) U of the sum of magnitudes; ex2.approx by 2^-22 of its result.
"""
import math

import torch

U = 2.0 ** -24
EX2 = 2.0 ** -22
TREE = 16  # levels of the widest tree of a block and a cluster, with their rebasing


def half(dtype):
    return torch.finfo(dtype).eps / 2


def excess(got, want, tol):
    """Largest error over its tolerance (at most 1 where all is well); equal
    infinities and NaN are no error."""
    most = torch.finfo(got.dtype).max
    got, want = got.double(), want.double()
    want = torch.where(want.abs() > most, want.sign() * math.inf, want)  # past the type's range
    same = (got == want) | (got.isnan() & want.isnan())
    off = (got - want).abs() / (tol + 1e-38)
    return torch.where(same, 0.0, torch.where(off.isnan(), math.inf, off)).max().item() if got.numel() else 0.0


# --- norm -------------------------------------------------------------------
def norm_terms(cols):
    """Sequential additions of a thread's sum of squares."""
    return 32 if cols <= 32768 else 32 * -(-cols // 32768)


def norm_fwd(x, residual, weight, eps, offset):
    """(h, y, rstd, relative error of y before it is rounded) from 32-bit h."""
    h = x.float() if residual is None else x.float() + residual.float()
    d = h.double()
    rstd = 1.0 / torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
    w = 1.0 if weight is None else weight.double() + offset
    return h, d * rstd * w, rstd[..., 0], (norm_terms(x.shape[-1]) + TREE) / 2 * U + 6 * U


def norm_bwd(dy, h, rstd, weight, dh, offset):
    """(d, its absolute tolerance, dweight, its tolerance) before rounding,
    from the stored h and rstd."""
    cols = h.shape[-1]
    dy, h, r = dy.double(), h.double(), rstd.double()[..., None]
    w = torch.ones(cols, dtype=torch.float64, device=h.device) if weight is None else weight.double() + offset
    u = dy * w
    b = r ** 3 * (u * h).mean(-1, keepdim=True)
    size = r ** 3 * (u * h).abs().mean(-1, keepdim=True)
    d = r * u - h * b + (0.0 if dh is None else dh.double())
    tol = U * (8 * ((r * u).abs() + (h * b).abs() + (0.0 if dh is None else dh.double().abs()))
               + (norm_terms(cols) + TREE + 6) * h.abs() * size)
    n = (dy * h * r).reshape(-1, cols)
    return d, tol, n.sum(0), (n.shape[0] + TREE + 4) * U * n.abs().sum(0)


# --- logits -----------------------------------------------------------------
class Rows:
    """Softmax statistics of rows of logits, 64 bits."""

    def __init__(self, logits, scale):
        z = logits.double()
        n = z.shape[1]
        top = z.max(1, keepdim=True).values if n else z.new_full((z.shape[0], 1), -math.inf)
        self.empty = (top == -math.inf)[:, 0]
        t = (z - torch.where(top == -math.inf, 0.0, top)) * scale
        e = torch.exp(t)
        l = e.sum(1, keepdim=True)
        safe = torch.where(l == 0, 1.0, l)
        self.t, self.p, self.log_l = t, e / safe, torch.log(safe)[:, 0]
        self.logp = torch.where(self.empty[:, None], -math.inf, t - torch.log(safe))
        pt = torch.where(e == 0, 0.0, self.p * t)
        self.U = -pt.sum(1)
        self.entropy = torch.where(self.empty, 0.0, self.log_l + self.U)
        terms = 8 + max(8, n // 8 // 512 + 1) + TREE
        self.l_tol = EX2 + (3 * self.U + terms) * U  # relative, of l
        square = torch.where(e == 0, 0.0, self.p * t * t).sum(1)
        self.u_tol = self.U * (EX2 + (terms + 4) * U + self.l_tol) + 3 * U * square
        self.logp_tol = self.l_tol[:, None] + 4 * U * (self.t.abs() + self.log_l[:, None])
        self.entropy_tol = self.l_tol + self.u_tol + 4 * U * (self.log_l + self.U)
        self.p_tol = EX2 + 4 * U + 3 * U * torch.where(e == 0, 0.0, t.abs()) + self.l_tol[:, None]  # relative


def logprobs(logits, tokens, scale):
    """(rows' statistics, which rows count, logprob, its tolerance)."""
    r = Rows(logits, scale)
    kept = (tokens >= 0) & (tokens < logits.shape[1])
    at = torch.where(kept, tokens, 0).long()[:, None]
    if logits.shape[1] == 0:
        zero = torch.zeros(logits.shape[0], dtype=torch.float64, device=logits.device)
        return r, kept, zero, zero
    lp = torch.where(kept, r.logp.gather(1, at)[:, 0], 0.0)
    return r, kept, lp, r.logp_tol.gather(1, at)[:, 0]


def top_of(logits, kept, top):
    """Columns of the `top` largest logits above -inf, -1 for none; equal ones
    by the lower column, NaN never."""
    z = torch.where(logits.isnan(), -math.inf, logits.double())
    order = torch.sort(z, dim=1, descending=True, stable=True)
    index = torch.where((order.values == -math.inf) | ~kept[:, None], -1, order.indices)[:, :top]
    return torch.nn.functional.pad(index, (0, top - index.shape[1]), value=-1)


def logprobs_bwd(r, kept, tokens, g, ge, scale):
    """(dz, tolerance) before rounding."""
    live = (kept & ~r.empty)[:, None]
    g = torch.zeros(r.p.shape[0], dtype=torch.float64, device=r.p.device)[:, None] if g is None else g.double()[:, None]
    ge = torch.zeros_like(g) if ge is None else ge.double()[:, None]
    t = torch.where(r.p == 0, 0.0, r.t)
    one = torch.zeros_like(r.p).scatter_(1, torch.where(kept, tokens, 0).long()[:, None], 1.0)
    d = scale * (g * one - r.p * (g + ge * (t + r.U[:, None])))
    size = scale * r.p * (g.abs() + ge.abs() * (t.abs() + r.U[:, None]))
    tol = size * (r.p_tol + 6 * U) + scale * r.p * ge.abs() * r.u_tol[:, None] + 4 * U * scale * g.abs() * one
    return torch.where(live, d, 0.0), tol


def distill(logits, index, teacher, scale, lse=None):
    """(rows' statistics, q, loss, its tolerance, relative tolerance of q)."""
    r = Rows(logits, scale)
    has = (index >= 0) & (index < logits.shape[1])
    at = torch.where(has, index, 0).long()
    score = torch.where(has, teacher.double() * scale, -math.inf)
    high = score.max(1, keepdim=True).values if score.shape[1] else score.new_full((score.shape[0], 1), -math.inf)
    high = torch.where(high == -math.inf, 0.0, high)
    total = torch.exp(score - high).sum(1, keepdim=True)
    norm = torch.log(torch.where(total == 0, 1.0, total)) if lse is None else lse.double()[:, None] - high
    logq = (score - high) - norm
    q = torch.exp(logq)
    far = torch.where(q == 0, 0.0, (score - high).abs())
    cancel = 0.0 if lse is None else 2 * U * (high.abs() + lse.double()[:, None].abs())
    q_tol = 2 * EX2 + (3 * far + teacher.shape[1] / 32 + TREE + 8) * U + cancel
    if logits.shape[1] == 0 or teacher.shape[1] == 0:
        zero = torch.zeros(logits.shape[0], dtype=torch.float64, device=logits.device)
        return r, q, zero, zero, q_tol
    logp = r.logp.gather(1, at)
    part = torch.where(q == 0, 0.0, q * (logq - logp))
    off = q_tol * (logq - logp).abs() + 4 * U * (logq.abs() + logp.abs() + far) + r.logp_tol.gather(1, at) + cancel
    tol = torch.where((q == 0) | ~off.isfinite(), 0.0, q * off).sum(1)
    tol = tol + (teacher.shape[1] / 32 + TREE) * U * torch.where(part.isfinite(), part.abs(), 0.0).sum(1)
    return r, q, part.sum(1), tol, q_tol


def distill_bwd(r, q, q_tol, index, g, scale, n):
    has = (index >= 0) & (index < n)
    at = torch.where(has, index, 0).long()
    g = g.double()[:, None] * scale
    Q = q.sum(1, keepdim=True)
    listed = torch.zeros_like(r.p).scatter_add_(1, at, torch.where(has, q, 0.0))
    d = g * (Q * r.p - listed)
    off = torch.zeros_like(r.p).scatter_add_(1, at, torch.where(has, q * (q_tol + q.shape[1] * U), 0.0))
    Q_tol = (q * q_tol).sum(1, keepdim=True) + (q.shape[1] / 32 + TREE) * U * Q
    tol = g.abs() * (Q * r.p * (r.p_tol + 8 * U) + r.p * Q_tol + off + 4 * U * listed)
    return torch.where(r.empty[:, None], 0.0, d), tol
