"""Rows of logits in which one token is nearly certain: its log probability,
the row's entropy and the given token's gradient are far below the logits'
spread, so whatever is subtracted to form them must be of their own size.

The bounds, in roundings u = 2^-24 of numbers relative to the row's largest
logit (d = z - max z, exp2 and log2 to 2u).  The largest entry adds exactly 1
to the sum S = 1 + R, R = sum of the other e^d.  What is added to a partial sum
that holds the 1 costs u of it each time: a thread's word and its words by
halves (at most 7), its chunks (at most 16), a wave (6), a block (3), a row's
segments (6): K = 38.  An e^d is off by (3 |d| + 2) u, its own sums by K u:
  S:      u (K + sum p (3 |d| + K + 2)),        relatively, p of the others
  log S:  that and 3u log S;
  log p:  that and 4u |d|;
  H = log S - sum p d: each p |d| is off by (3 |d| + 2 K + 4) u, its sums K u.
With 1 - p the others' sum of p (m0), mean |d| m1 and mean d^2 m2 this is
  log p_t:  u (K + (K + 2) m0 + 3 m1 + 4 |log p_t| + 4 |d_t|)
  H:        u (K + (K + 2) m0 + (3 K + 9) m1 + 3 m2 + 4 H).
The given token's gradient gl (1 - p) / T is off by gl (p tol(log p) +
4u (1 - p)) / T and half a step of its type."""
import math

import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
U, K = P.U, 38
# cut rows, whole rows in short and long chunks, rows in registers of 4 and 8 waves, streamed rows
SIZES = [(3, 128256), (4, 300001), (5, 1000), (7, 9000), (40, 16000), (6, 32000), (300, 12301), (300, 32000), (200, 50257), (300, 131073)]


def draw(rows, vocab, dtype, seed, temperature):
    """One token 8 to 16 nats above the others' middle, in the row's later two thirds; the given token by
    turns that one and any other."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * 0.7
    at = torch.randint(vocab // 3, vocab, (rows,), generator=g)
    x[torch.arange(rows), at] = 8.0 + 8.0 * torch.rand(rows, generator=g)
    t = at.clone()
    t[1::4] = torch.randint(0, vocab, (len(t[1::4]),), generator=g)
    return (x * temperature).to(dtype).cuda(), at.cuda(), t.cuda(), g


def expected(x, t, temperature):
    z = x.double() / temperature
    top = z.amax(1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    p = e / s
    best = d == 0
    m0 = torch.where(best, 0.0, p).sum(1)
    m1, m2 = (p * d.abs()).sum(1), (p * d * d).sum(1)
    dt = d.gather(1, t[:, None]).squeeze(1)
    lp = dt - torch.log(s.squeeze(1))
    ent = torch.log(s.squeeze(1)) + m1
    base = K + (K + 2) * m0
    ltol = U * (base + 3 * m1 + 4 * lp.abs() + 4 * dt.abs())
    etol = U * (base + (3 * K + 9) * m1 + 3 * m2 + 4 * ent)
    return lp, ltol, ent, etol


def within(got, ref, tol, what):
    off = (got.double() - ref).abs() / tol
    assert bool((off <= 1).all()), f"{what}: {off.max().item():.2f} of the bound at {int(off.argmax())}, {int((off > 1).sum())} rows"


@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_one_token_nearly_certain(rows, vocab, dtype, temperature):
    x, at, t, g = draw(rows, vocab, dtype, rows + vocab, temperature)
    lp, ltol, ent, etol = expected(x, t, temperature)
    gl = (torch.rand(rows, generator=g) + 0.5).cuda()
    best, btol, _, _ = expected(x, at, temperature)
    forms = []
    for top in (0, 3):
        r = L.token_logprobs(x, t, top=top, temperature=temperature)
        forms.append((f"forward, top {top}", r.logprob, r.entropy))
        if top:
            assert torch.equal(r.top_id[:, 0], at)
            within(r.top_logprob[:, 0], best, btol, "the best entry")
            assert bool((r.top_logprob <= 0).all())
    xg = x.clone().requires_grad_()
    r = L.token_logprobs(xg, t, temperature=temperature)
    auto, = torch.autograd.grad(r.logprob, xg, gl)
    forms.append(("with a graph", r.logprob.detach(), r.entropy.detach()))
    one = L.token_logprobs_grad(x, t, gl, temperature=temperature)
    both = L.token_logprobs_grad(x, t, gl, torch.zeros_like(gl), temperature=temperature)
    forms += [("with the gradient", one.logprob, one.entropy), ("with both gradients", both.logprob, both.entropy)]
    for name, a, b in forms:
        within(a, lp, ltol, name + ", log probability")
        within(b, ent, etol, name + ", entropy")
        assert bool((a <= 0).all()) and bool((b >= 0).all()), name
    p = torch.exp(lp)
    want = gl.double() * -torch.expm1(lp) / temperature
    tol = gl.double() * (p * ltol + 4 * U * -torch.expm1(lp)) / temperature
    tol = tol + P.half_step(dtype) * (want.abs() + tol) + 4 * U * want.abs() + P.smallest(dtype)
    for name, grad in (("graph", auto), ("one call", one.grad), ("with the entropy's", both.grad)):
        within(grad.gather(1, t[:, None]).squeeze(1), want, tol, name + ", the given token's gradient")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(3, 128256), (5, 1000), (6, 32000), (300, 32000), (300, 131073)])
def test_entropy_gradient_of_the_likely_token(rows, vocab, dtype):
    """-gh p (log p + H) of the likely token: both terms are near 0 and each is off by its own bound."""
    x, at, _, g = draw(rows, vocab, dtype, 3 * rows + vocab, 1.0)
    lp, ltol, ent, etol = expected(x, at, 1.0)
    gh = (torch.rand(rows, generator=g) + 0.5).cuda()
    want = -gh.double() * torch.exp(lp) * (lp + ent)
    tol = gh.double() * (ltol + etol + 4 * U * (lp.abs() + ent)) + U * 40 * want.abs()
    tol = tol + P.half_step(dtype) * (want.abs() + tol) + P.smallest(dtype)
    xg = x.clone().requires_grad_()
    auto, = torch.autograd.grad(L.token_logprobs(xg).entropy, xg, gh)
    zero, none = torch.zeros_like(gh), torch.full_like(at, -100)
    one = L.token_logprobs_grad(x, none, zero, gh).grad
    for name, grad in (("graph", auto), ("one call", one)):
        within(grad.gather(1, at[:, None]).squeeze(1), want, tol, name)


@pytest.mark.parametrize("vocab", [1000, 32000, 131073])
@pytest.mark.parametrize("rows", [2, 300])
def test_two_tokens_share_the_row(rows, vocab):
    """Two equal logits far above the rest, in any two places: log p = -log 2 and H = log 2 but for the rest."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g) * 0.5
    two = torch.stack([torch.randperm(vocab - vocab // 3, generator=g)[:2] + vocab // 3 for _ in range(rows)])
    x.scatter_(1, two, 15.0)
    x, t = x.to(torch.bfloat16).cuda(), two[:, 1].cuda()
    lp, ltol, ent, etol = expected(x, t, 1.0)
    assert bool(((lp + math.log(2)).abs() < 0.1).all())
    r = L.token_logprobs(x, t, top=2)
    within(r.logprob, lp, ltol, "log probability")
    within(r.entropy, ent, etol, "entropy")
    one = L.token_logprobs_grad(x, t, torch.ones(rows, device="cuda"))
    within(one.logprob, lp, ltol, "log probability, one call")
    within(one.entropy, ent, etol, "entropy, one call")
