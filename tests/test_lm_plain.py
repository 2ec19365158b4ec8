"""The plain 64-bit forms of the language-model operators (lm_plain.py)
against torch's own functions and automatic differentiation in 64 bits."""
import math

import torch

import lm_plain as P


def test_logprob_forms():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 40, generator=g).double() * 3
    x[2, :20] = -math.inf
    x[4] = -math.inf
    t = torch.tensor([3, -100, 25, 40, 0])
    lp, tol, en, et = P.logprob(x, t, 1.3)
    ref = torch.log_softmax(x / 1.3, 1)
    assert abs(lp[0] - ref[0, 3]) < 1e-12 and lp[1] == 0 and abs(lp[2] - ref[2, 25]) < 1e-12 and lp[3] == 0
    assert lp[4] == -math.inf and en[4] == 0
    dist = torch.distributions.Categorical(logits=x[[0, 1, 3]] / 1.3)
    assert (en[[0, 1, 3]] - dist.entropy()).abs().max() < 1e-12
    assert bool((tol < 1e-4).all()) and bool((et < 1e-3).all())
    y = x[:4].clone().clamp_min(-60).requires_grad_()
    gl, gh = torch.randn(4, generator=g).double(), torch.randn(4, generator=g).double()
    z = torch.log_softmax(y / 1.3, 1)
    f = gl[0] * z[0, 3] + gl[2] * z[2, 25] + (gh * -(torch.exp(z) * z).sum(1)).sum()
    auto, = torch.autograd.grad(f, y)
    grad, _ = P.logprob_grad(y.detach(), t[:4], gl, gh, 1.3)
    assert (grad - auto).abs().max() < 1e-10


def test_distill_forms():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(3, 30, generator=g).double() * 2).requires_grad_()
    ids = torch.tensor([[1, 5, 9], [2, 2, 7], [0, -1, 30]])
    t = torch.log(torch.tensor([[0.5, 0.2, 0.1], [0.3, 0.2, 0.4], [0.6, 0.3, 0.05]]).double())
    up = torch.randn(3, generator=g).double()
    lp = torch.log_softmax(x / 0.8, 1)
    for tail in (False, True):
        rows = []
        for r in range(3):
            use = [k for k in range(3) if 0 <= ids[r, k] < 30]
            q = torch.exp(t[r, use])
            if not tail:
                q = q / q.sum()
            f = (q * (torch.log(q) - lp[r, ids[r, use]])).sum()
            if tail:
                rest = [j for j in range(30) if j not in ids[r].tolist()]
                left = 1 - q.sum()
                f = f + left * (torch.log(left) - torch.logsumexp(lp[r, rest], 0))
            rows.append(f)
        loss = torch.stack(rows)
        auto, = torch.autograd.grad((loss * up).sum(), x, retain_graph=True)
        a, _, b, _ = P.distill(x.detach(), ids, t, tail, 0.8, up)
        assert (a - loss).abs().max() < 1e-12
        assert (b - auto).abs().max() < 1e-12


def test_rows_in_8_bits():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, -126.5], [0.0, 0, 0, 0, 0]])
    q, s = P.row_codes(x)
    assert q.tolist() == [[127, 0, 2, -2, -126], [0, 0, 0, 0, 0]] and s.tolist() == [1.0, 0.0]
