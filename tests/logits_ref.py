"""Plain float64 forms of the operators on the streams' logits, and how far a float32
computation of them may be off. Any device; logits [S, n, V] (or [S, V], as n = 1).

Tolerances. u = 2^-24 is half a float32 step. With d_i = x_i - max: the exponent c d_i takes
three roundings (the difference, c log2 e, the product), the 2^x instruction is within 2 ulp
(2^-22), and s is summed in float32 by at least 32 threads: a term meets at most
V / 256 + 96 additions. Hence, with A1 = sum p |c d|, A2 = sum p (c d)^2,
    s within a relative  es = (V / 256 + 96) u + 2^-22 + 3 u A1,
    ln s within          tl = es + 2 u |ln s|,
    lse                  tl + 2 u (|c m| + |lse|),
    ln p_i               tl + 3 u |c d_i| + 2 u |ln p_i|,
    entropy              tl + 3 u A2 + A1 (2^-22 + (V / 256 + 99) u + es) + 2 u H
(the terms of w all have one sign). Gradients multiply such factors; a bf16 result adds half
a step, 2^-8 of its value (float32: 2^-24). Probabilities below 2^-126 may be flushed."""
import math

import torch

U = 2.0 ** -24
EX2 = 2.0 ** -22
TINY = 2.0 ** -120


def rows3(x):
    return x if x.dim() == 3 else x.unsqueeze(1)


class Row:
    """Statistics of logits x [S, n, V] (any float type) in float64, with their tolerances."""

    def __init__(self, x, c, keep=None):
        x = rows3(x).double()
        V = x.shape[-1]
        if keep is not None:
            x = torch.where(keep, x, -math.inf)
        self.x, self.c = x, c
        m = x.amax(-1, keepdim=True)
        self.none = m.squeeze(-1) == -math.inf
        self.m = torch.where(m == -math.inf, 0.0, m)
        cd = c * (x - self.m)
        e = cd.exp()
        s = e.sum(-1, keepdim=True)
        self.ln_s = s.log()
        self.lse = c * self.m + self.ln_s
        self.logp = cd - self.ln_s
        self.p = torch.where(self.none.unsqueeze(-1), 0.0, e / s)
        z = torch.where(self.p > 0, cd, 0.0)
        self.a1 = (self.p * z.abs()).sum(-1, keepdim=True)
        a2 = (self.p * z * z).sum(-1, keepdim=True)
        adds = V / 256 + 96
        es = adds * U + EX2 + 3 * U * self.a1
        ln_s = torch.where(torch.isfinite(self.ln_s), self.ln_s, 0.0).abs()
        lse = torch.where(torch.isfinite(self.lse), self.lse, 0.0).abs()
        self.t_ln = es + 2 * U * ln_s
        self.t_lse = self.t_ln + 2 * U * ((c * self.m).abs() + lse)
        self.t_logp = self.t_ln + 3 * U * cd.abs() + 2 * U * (cd - ln_s).abs()
        self.entropy = torch.where(self.none.unsqueeze(-1), 0.0, self.ln_s + self.a1)
        self.entropy = torch.where(torch.isnan(s), math.nan, self.entropy)
        self.t_entropy = (self.t_ln + 3 * U * a2 + self.a1 * (EX2 + (adds + 3) * U + es)
                          + 2 * U * self.entropy.abs())
        self.rel_p = 3 * U * z.abs() + EX2 + es + 4 * U


def targets(tokens, V, pad):
    """(there, index) of tokens [S, n]."""
    there = (tokens >= 0) & (tokens < V) & (tokens != pad)
    return there, torch.where(there, tokens, 0).long().unsqueeze(-1)


def logprob(x, tokens, pad=-1, c=1.0):
    """{name: (value, tolerance)} of logprob, entropy and lse [S, n]."""
    r = Row(x, c)
    out = {"entropy": (r.entropy.squeeze(-1), r.t_entropy.squeeze(-1)),
           "lse": (torch.where(r.none, -math.inf, r.lse.squeeze(-1)), r.t_lse.squeeze(-1))}
    if tokens is not None:
        there, at = targets(tokens.reshape(r.none.shape), r.x.shape[-1], pad)
        lp, t = r.logp.gather(-1, at).squeeze(-1), r.t_logp.gather(-1, at).squeeze(-1)
        lp = torch.where(r.none, -math.inf, lp)
        out["logprob"] = (torch.where(there, lp, 0.0), torch.where(there, t, 0.0))
    return out


def top(x, k, c=1.0):
    """(ids, logprob, tolerance) [S, n, k] of the k most likely tokens by a stable sort."""
    r = Row(x, c)
    V = r.x.shape[-1]
    broken = torch.isnan(r.lse.squeeze(-1)) | (r.x == math.inf).any(-1)
    order = torch.sort(torch.nan_to_num(r.x, nan=-math.inf, posinf=math.inf, neginf=-math.inf),
                       dim=-1, descending=True, stable=True)
    ids, values = order.indices[..., :k], order.values[..., :k]
    lp = r.logp.gather(-1, ids)
    t = r.t_logp.gather(-1, ids)
    ids = torch.where(values == -math.inf, -1, ids)
    lp = torch.where(values == -math.inf, -math.inf, lp)
    if k > V:
        more = (*ids.shape[:-1], k - V)
        ids = torch.cat([ids, ids.new_full(more, -1)], -1)
        lp = torch.cat([lp, lp.new_full(more, -math.inf)], -1)
        t = torch.cat([t, t.new_zeros(more)], -1)
    ids = torch.where(broken.unsqueeze(-1), -1, ids)
    lp = torch.where(broken.unsqueeze(-1), math.nan, lp)
    return ids, lp, t


def rounding(value, dtype):
    return value.abs() * torch.finfo(dtype).eps / 2 + TINY


def logprob_grad(x, tokens, a=None, b=None, z=None, pad=-1, c=1.0):
    """(dlogits, tolerance) [S, n, V]; a, b, z: upstream of logprob, entropy, lse [S, n]."""
    r = Row(x, c)
    zero = torch.zeros(r.none.shape, dtype=torch.float64, device=r.x.device)
    a, b, z = (zero if v is None else v.reshape(zero.shape).double() for v in (a, b, z))
    hot = torch.zeros_like(r.x)
    if tokens is not None:
        there, at = targets(tokens.reshape(zero.shape), r.x.shape[-1], pad)
        a = torch.where(there, a, 0.0)
        hot.scatter_(-1, at, there.double().unsqueeze(-1))
    off = (r.none | ((a == 0) & (b == 0) & (z == 0))).unsqueeze(-1)
    a, b, z = a.unsqueeze(-1), b.unsqueeze(-1), z.unsqueeze(-1)
    lp = torch.where(r.p > 0, r.logp, 0.0)
    coef = (z - a) - b * (lp + r.entropy)
    d = c * (r.p * coef + a * hot)
    size = z.abs() + a.abs() + b.abs() * (lp.abs() + r.entropy + r.ln_s.abs())
    t = c * r.p * (r.rel_p * coef.abs() + b.abs() * (r.t_entropy + 2 * r.t_ln
                                                     + 3 * U * lp.abs()) + 8 * U * size)
    t = t + c * 4 * U * a.abs() * hot
    d, t = torch.where(off, 0.0, d), torch.where(off, 0.0, t)
    dt = x.dtype
    return d, t + rounding(d.abs() + t, dt)


def distill(x, ids, teacher, g=None, tail=False, c=1.0):
    """(loss, tolerance, dlogits, tolerance) for lists ids, teacher [S, n, k]."""
    dt = x.dtype
    all_ = Row(x, c)
    V = all_.x.shape[-1]
    lead = all_.none.shape
    k = ids.shape[-1]
    ids = ids.reshape(*lead, k).long()
    there = (ids >= 0) & (ids < V)
    t = torch.where(there, teacher.reshape(ids.shape).double(), -math.inf)
    at = torch.where(there, ids, 0)
    has = there.any(-1)
    if tail:
        q = t.exp()
        lq = t
        e_lq = torch.zeros_like(t)
    else:
        has = has & ~(t == -math.inf).all(-1)
        safe = torch.where(has.unsqueeze(-1), t, 0.0)
        tm = safe.amax(-1, keepdim=True)
        lq = safe - torch.logsumexp(safe, -1, keepdim=True)
        q = torch.where(there, lq.exp(), 0.0)
        e_lq = 3 * U * ((safe - tm).abs() + lq.abs()) + (k + 6) * U
        e_lq = torch.where(q == 0, 0.0, e_lq)
    inside = torch.zeros_like(all_.x).scatter_add_(-1, at, there.double()) > 0
    rel_q = e_lq + 4 * U
    lp = torch.where(all_.none.unsqueeze(-1), -math.inf, all_.logp.gather(-1, at))
    t_lp = all_.t_logp.gather(-1, at)
    live = ~(q == 0)
    gap = torch.where(live, lq - lp, 0.0)
    terms = torch.where(live, q * gap, 0.0)
    loss = terms.sum(-1)
    t_loss = torch.where(live, q * (gap.abs() * rel_q + e_lq + t_lp), 0.0).sum(-1)
    t_loss = t_loss + (k + 4) * U * torch.nan_to_num(terms.abs()).sum(-1)
    soft = torch.zeros_like(all_.x)
    qr = torch.zeros(lead, dtype=torch.float64, device=all_.x.device)
    rel_rest = torch.zeros_like(all_.x)
    if tail:
        rest = Row(x, c, keep=~inside)
        qr = torch.where(has & ~rest.none, (1.0 - q.sum(-1)).clamp_min(0.0), 0.0)
        lr = (c * (rest.m - all_.m) + rest.ln_s - all_.ln_s).squeeze(-1)
        lr = torch.where(rest.none, 0.0, lr)
        some = qr > 0
        lnq = torch.where(some, qr.log(), 0.0)
        term = torch.where(some, qr * (lnq - lr), 0.0)
        loss = loss + term
        t_r = (rest.t_ln + all_.t_ln).squeeze(-1) + 4 * U * (lr.abs() + lnq.abs() + 1) \
            + 4 * U * (c * (rest.m - all_.m)).abs().squeeze(-1) \
            + 2 * U * (rest.ln_s.abs() + all_.ln_s.abs()).squeeze(-1).nan_to_num(0, 0, 0)
        t_loss = t_loss + torch.where(some, qr * t_r, 0.0) + 4 * U * term.abs() \
            + k * 2.0 ** -50 * (1 + lnq.abs() + lr.abs())  # q_r is 1 - a float64 sum
        soft, rel_rest = rest.p, rest.rel_p
    loss, t_loss = torch.where(has, loss, 0.0), torch.where(has, t_loss, 0.0)
    t_loss = torch.nan_to_num(t_loss, 0, 0, 0) + U * torch.nan_to_num(loss.abs(), 0, 0, 0)
    Q = torch.where(torch.isnan(q).any(-1), math.nan, q.sum(-1) + qr).unsqueeze(-1)
    g = torch.ones(lead, dtype=torch.float64, device=qr.device) if g is None \
        else g.reshape(lead).double()
    gc = (g * c).unsqueeze(-1)
    want = torch.zeros_like(all_.x).scatter_add_(-1, at, torch.where(there, q, 0.0))
    t_want = torch.zeros_like(all_.x).scatter_add_(-1, at, torch.where(there, q * rel_q, 0.0))
    qr = qr.unsqueeze(-1)
    d = gc * (Q * all_.p - want - qr * soft)
    t_d = gc.abs() * (Q * all_.p * (all_.rel_p + (k + 6) * U) + t_want + (k + 4) * U * want
                      + qr * soft * (rel_rest + 6 * U) + k * 2.0 ** -50 * (soft + all_.p))
    off = (~has | (g == 0) | all_.none).unsqueeze(-1)
    d, t_d = torch.where(off, 0.0, d), torch.where(off, 0.0, t_d)
    return loss, t_loss, d, t_d + rounding(d.abs() + t_d, dt)


def near(got, want, tol, what=""):
    """|got - want| <= tol where want is finite; the same infinity or NaN elsewhere."""
    got = got.double().reshape(want.shape)
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * math.inf, want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd]), f"{what}: infinities differ"
    assert torch.isfinite(got[fine]).all(), f"{what}: not finite"
    off = (got - want).abs()[fine] - tol.expand(want.shape)[fine]
    assert off.numel() == 0 or off.max().item() <= 0, \
        f"{what}: {off.max().item():.3g} past the tolerance"
