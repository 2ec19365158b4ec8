"""Distillation without a tail from lists whose numbers are not log probabilities near 0: q is e^t over
its sum, so a list means the same wherever it lies (ids that the student chose, low temperatures,
scores that were never normalised).  Against the plain 64-bit form and its tolerances (lm_plain.py),
which bound q by the normalised logarithms."""
import math

import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def near(got, ref, tol, dtype=torch.float32):
    half = P.half_step(dtype)
    lim = tol * (1 + half) + half * ref.abs() + P.smallest(dtype) + P.TINY
    off = (got.double().cpu() - ref).abs()
    assert bool((off <= lim).all()), f"{(off / lim).max().item():.3g} of the bound"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(2, 1000), (3, 150001), (300, 9000)])
@pytest.mark.parametrize("base", [0.0, -100.0, -207.0, -210.0, -300.0, -5000.0, 80.0, 400.0, -2.0 ** 25, 2.0 ** 25])
def test_a_list_means_the_same_wherever_it_lies(rows, vocab, dtype, base):
    g = torch.Generator().manual_seed(rows + vocab)
    x = (torch.randn(rows, vocab, generator=g) * 2).to(dtype)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:9] for _ in range(rows)])
    step = 4.0 if abs(base) > 1e6 else 0.25                # multiples that binary32 holds there
    t = base - step * torch.randint(0, 12, (rows, 9), generator=g).float()
    t[0, 4] = -math.inf                                    # the teacher excludes one
    ids[-1, 3] = -100                                      # and one is skipped
    up = torch.randn(rows, generator=g)
    for temp in (1.0, 0.5):
        a, at, b, bt = P.distill(x, ids, t, False, temp, up)
        xc, ic, tc, uc = x.cuda(), ids.cuda(), t.cuda(), up.cuda()
        loss, grad = L.distill_grad(xc, ic, tc, uc, tail=False, temperature=temp)
        near(loss, a, at)
        near(grad, b, bt, dtype)
        xg = xc.clone().requires_grad_()
        lo = L.distill_loss(xg, ic, tc, tail=False, temperature=temp)
        near(lo.detach(), a, at)
        got, = torch.autograd.grad(lo, xg, uc)
        near(got, b, bt, dtype)
        loss2, _ = L.distill_grad(xc, ic, tc, uc, tail=False, temperature=temp, inplace=True)
        assert torch.equal(loss2, loss) and torch.equal(xc, grad)


def test_lists_without_a_distribution():
    """Nothing but -inf: no teacher, loss and gradient 0; NaN and +inf: the row's results are NaN."""
    x = torch.randn(4, 500, generator=torch.Generator().manual_seed(1)).cuda()
    ids = torch.arange(5).repeat(4, 1).cuda()
    t = torch.full((4, 5), -1.0)
    t[0] = -math.inf
    t[1, 2] = math.nan
    t[2, 3] = math.inf
    for tail in (False, True):
        loss, grad = L.distill_grad(x, ids, t.cuda(), torch.ones(4, device="cuda"), tail=tail)
        assert bool(torch.isnan(loss[1:3]).all()) or tail  # (e^inf with a tail is an infinite q)
        assert bool(torch.isfinite(loss[3])) and bool(torch.isfinite(grad[3]).all())
        if not tail:
            assert loss[0].item() == 0 and bool((grad[0] == 0).all())
        xg = x.clone().requires_grad_()
        lo = L.distill_loss(xg, ids, t.cuda(), tail=tail)
        got, = torch.autograd.grad(lo.sum(), xg)
        assert torch.equal(lo.detach().nan_to_num(7.0), loss.nan_to_num(7.0))
        assert torch.equal(got[[0, 3]], grad[[0, 3]])
