"""Plain 64-bit forms of the language-model operators, in torch, with the
error each binary32 result of the library may have.

The bounds count roundings of u = 2^-24 (a binary32 operation; the hardware
exp2 and log2 2u).  With d = z_j - max z: an exponential e^d is off by
(3 |d| + 2) u relatively (difference, factor, product, exp2); a sum of
positive terms by at most 100 u more (at most 64 + 8 additions per thread, a
tree, a join of chunks).  A mean of terms over p is bounded with the means of
|d| and d^2 under p.  Results in 16 bits add half a step of their type.  The
hardware exp2 gives 0 below 2^-126 (TINY), so a gradient, an exponential times a
factor, may also be off by TINY times that factor."""
import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def smallest(t: torch.dtype) -> float:
    """Half the smallest subnormal step."""
    return {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[t]


def dist(x, temperature):
    """(z - max, log p, p, mean |d|, mean d^2) of rows with a distribution;
    rows of -inf alone give p = 0."""
    z = x.double() / temperature
    m = z.amax(1, keepdim=True)
    empty = m == -math.inf
    d = z - torch.where(empty, 0.0, m)
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    logp = d - torch.where(empty, 0.0, torch.log(s))
    p = torch.where(empty, 0.0, e / s)
    fin = torch.where(p > 0, d, 0.0)
    return d, logp, p, (p * fin.abs()).sum(1), (p * fin * fin).sum(1), empty.squeeze(1)


def lse_tol(m1):
    """log S: the exponentials' errors in the mean, the sum, the log."""
    return U * (110 + 3 * m1)


def logprob(x, targets, temperature):
    """(logprob, its tolerance, entropy, its tolerance)"""
    d, logp, p, m1, m2, empty = dist(x, temperature)
    vocab = x.shape[1]
    given = (targets >= 0) & (targets < vocab)
    at = torch.where(given, targets, 0)[:, None]
    lp = torch.where(given, logp.gather(1, at).squeeze(1), 0.0)
    dt = d.gather(1, at).squeeze(1).abs()
    tol = torch.where(given & torch.isfinite(dt), lse_tol(m1) + U * (4 * dt + 4 * lp.abs()), 0.0)
    ent = -torch.where(p > 0, p * logp, 0.0).sum(1)
    etol = lse_tol(m1) + U * (3 * m2 + 210 * m1 + 4 * ent.abs())
    return lp, tol, ent, torch.where(empty, 0.0, etol)


def top(x, k):
    """ids of the k largest, equal ones by lowest id"""
    return torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :k]


def logprob_grad(x, targets, gl, gh, temperature):
    """(gradient, tolerance before the type's rounding)"""
    d, logp, p, m1, m2, empty = dist(x, temperature)
    vocab, rows = x.shape[1], x.shape[0]
    given = (targets >= 0) & (targets < vocab) & ~empty
    gl = torch.where(given, gl.double(), 0.0) if gl is not None else torch.zeros(rows, device=x.device).double()
    gh = gh.double() if gh is not None else torch.zeros(rows, device=x.device).double()
    lpf = torch.where(p > 0, logp, 0.0)
    ent = -(p * lpf).sum(1)
    a = (-gl - gh * ent)[:, None]
    grad = p * (a - gh[:, None] * lpf)
    grad[torch.arange(rows, device=x.device)[given], targets[given]] += gl[given]
    # p's relative error, and the absolute one of the factor (H and log p)
    df = torch.where(p > 0, d, 0.0).abs()
    rel = lse_tol(m1)[:, None] + U * (4 * df + 8)
    factor = gl.abs()[:, None] + gh.abs()[:, None] * (ent[:, None] + lpf.abs())
    ftol = gh.abs()[:, None] * (lse_tol(m1) + U * (3 * m2 + 210 * m1 + 8 * ent))[:, None] \
        + gh.abs()[:, None] * rel + 6 * U * factor
    lost = TINY * (gl.abs() + gh.abs() * (ent + 90))[:, None]                # |log p| <= 88 there
    tol = p * (rel * factor + ftol) + 4 * U * grad.abs() + lost
    return grad / temperature, tol / temperature


def distill(x, ids, t, tail, temperature, g=None):
    """(loss, tolerance, gradient, tolerance before the type's rounding)"""
    d, logp, p, m1, m2, empty = dist(x, temperature)
    rows, vocab = x.shape
    ok = (ids >= 0) & (ids < vocab)
    at = torch.where(ok, ids, 0)
    td = torch.where(ok, t.double(), -math.inf)
    if not tail:
        norm = torch.logsumexp(td, 1, keepdim=True)
        td = torch.where(norm > -math.inf, td - norm, -math.inf)
    q = torch.exp(td)
    on = ok.any(1) & ~empty
    lp = logp.gather(1, at)
    listed = torch.zeros(rows, vocab, dtype=torch.bool, device=x.device)
    listed[torch.arange(rows, device=x.device)[:, None].expand_as(ids)[ok], ids[ok]] = True
    P = torch.where(listed, 0.0, p).sum(1)
    rest_lse = torch.logsumexp(torch.where(listed, -math.inf, logp), 1)     # log P, also where P underflows
    Q = q.sum(1)
    r = (1.0 - Q).clamp_min(0.0) if tail else torch.zeros(rows, device=x.device).double()
    has_rest = rest_lse > -math.inf
    r = torch.where(has_rest, r, 0.0)
    terms = torch.where(q > 0, q * (td - lp), 0.0)
    loss = terms.sum(1) + torch.where(r > 0, r * (torch.log(r.clamp_min(1e-300)) - rest_lse), 0.0)
    loss = torch.where(on, loss, 0.0)
    # each term q (log q - log p): q off by (6|t| + 4)u, the logs by (4|t| + 4|lp|)u and log S
    tf, lf = torch.where(q > 0, td, 0.0).abs(), torch.where(q > 0, lp, 0.0).abs()
    lf = torch.where(torch.isfinite(lf), lf, 0.0)
    qtol = q * U * (6 * tf + 10)                                            # of one q_k
    tol = (qtol * (tf + lf) + q * (U * (6 * tf + 6 * lf) + lse_tol(m1)[:, None])).sum(1) \
        + 70 * U * terms.abs().nan_to_num(0.0, 0.0, 0.0).sum(1)
    rtol = qtol.sum(1) + 70 * U * (1 + Q)                                   # of r
    lnr = torch.log(r.clamp_min(U)).abs()
    lnP = torch.where(has_rest, rest_lse, 0.0).abs()
    if tail:
        tol = tol + torch.where(has_rest, rtol * (lnr + lnP + 1) + r * (lse_tol(m1) * 2 + U * (120 + 6 * lnP)), 0.0)
    if g is None:
        return loss, tol
    w = torch.where(on, g.double(), 0.0)[:, None]
    qr = (Q + r)[:, None]
    # the entries' shares of the rest, from the rest's own largest (far below 1 where P underflows)
    rest = torch.where(listed, -math.inf, x.double() / temperature)
    share = torch.where(has_rest[:, None], torch.softmax(rest, 1), 0.0)
    qsum = torch.zeros(rows, vocab, dtype=torch.float64, device=x.device)
    qsum.scatter_add_(1, at, torch.where(ok, q, 0.0))
    grad = w * (qr * p - qsum - r[:, None] * share)
    df = torch.where(p > 0, d, 0.0).abs()
    rel = 2 * lse_tol(m1)[:, None] + U * (8 * df + 130)
    qst = torch.zeros(rows, vocab, dtype=torch.float64, device=x.device)
    qst.scatter_add_(1, at, torch.where(ok, qtol, 0.0))
    gtol = w.abs() * (qr * p * rel + qst + 70 * U * qsum + share * ((rtol * 2 + 4 * U)[:, None]
                      + (r[:, None] + qr * P[:, None]) * rel) + TINY * (2 * qr + r[:, None])) + 4 * U * grad.abs()
    return loss, tol, grad / temperature, gtol / temperature


def row_codes(x):
    """(codes, scale in binary32) of rows of finite values"""
    v = x.double()
    a = v.abs().amax(1, keepdim=True)
    q = torch.where(a > 0, torch.round(v * 127.0 / torch.where(a > 0, a, 1.0)), 0.0)
    return q.to(torch.int8), (a.squeeze(1).float() / 127.0)


def int8_product(qa, sa, qb, sb, bias, dtype):
    """(out, tolerance) with out in 64 bits"""
    acc = qa.double() @ qb.double().t()
    y = acc * sa.double()[:, None] * sb.double()[None]
    tol = 4 * U * y.abs()
    if bias is not None:
        y = y + bias.double()[None]
    tol = tol + (U + half_step(dtype)) * y.abs() * (1 + 8 * U) + smallest(dtype) + tol * half_step(dtype)
    return y, tol
