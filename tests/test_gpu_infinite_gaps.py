"""Preferences between sequences of which one is impossible: the gap d is infinite, and the loss
(1 - smoothing) log(1 + e^-d) + smoothing log(1 + e^d) and its slope have their limits there, 0 or infinity
for each term of a weight above 0; a term of weight 0 is not there."""
import math

import pytest
import torch

from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu
INF = math.inf


def limit(d, smoothing):
    """(loss, its slope in d)"""
    less, more = (0.0, INF) if d > 0 else (INF, 0.0)               # log(1 + e^-d), log(1 + e^d)
    loss = sum(w * t for w, t in ((1 - smoothing, less), (smoothing, more)) if w > 0)
    return loss, smoothing if d > 0 else smoothing - 1


# many tokens of few pairs: several blocks share a pair
@pytest.mark.parametrize("length", [1, 5, 700, 30000])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("smoothing", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("side,beta", [(0, 0.5), (1, 0.5), (0, -0.5), (1, -0.5)])
def test_an_impossible_sequence(length, average, smoothing, side, beta):
    g = torch.Generator().manual_seed(length)
    lp = -torch.rand(4 * length, generator=g)
    lp[side * length + length // 2] = -INF                         # pair 0; pair 1 is an ordinary one
    offsets = (torch.arange(5) * length).cuda()
    d = -INF if (side == 0) == (beta > 0) else INF
    x = lp.cuda().requires_grad_()
    r = L.preference_loss(x, offsets, beta=beta, smoothing=smoothing, average=average)
    loss, slope = limit(d, smoothing)
    assert r.loss[0].item() == loss and bool(r.loss[1].isfinite())
    grad, = torch.autograd.grad(r.loss.sum(), x)
    each = slope * beta / (length if average else 1)
    want = torch.full((length,), each)
    assert torch.equal(grad[:length].cpu(), want) and torch.equal(grad[length:2 * length].cpu(), -want)
    assert bool(grad[2 * length:].isfinite().all()) and bool(grad[2 * length:].any())
    # the reference's impossible token: the other way round
    y = torch.zeros(4 * length).cuda()
    r = L.preference_loss(y, offsets, lp.cuda(), beta=beta, smoothing=smoothing, average=average)
    assert r.loss[0].item() == limit(-d, smoothing)[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("vocab", [60, 40000, 140000])
@pytest.mark.parametrize("inplace", [False, True])
def test_an_impossible_token_of_logits(dtype, vocab, inplace):
    """The rejected sequence's token is masked: the pair is certain, its loss 0 and without a gradient; the
    chosen one's: the loss is infinite, its gradient is not."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(8, vocab, generator=g).to(dtype)
    t = torch.randint(0, vocab, (8,), generator=g)
    x[3, t[3]] = -INF                                              # rejected of pair 0
    x[4, t[4]] = -INF                                              # chosen of pair 1
    r = L.preference_grad(x.cuda(), t.cuda(), torch.tensor([0, 2, 4, 6, 8]).cuda(), beta=0.5, inplace=inplace)
    assert r.loss.tolist() == [0.0, INF]
    assert r.reward[0, 1].item() == -INF and r.reward[1, 0].item() == -INF
    assert not r.grad[:4].any() and bool(r.grad[4:].isfinite().all()) and bool(r.grad[4:].any(1).all())
    p = torch.softmax(x[4:].double(), 1)
    up = torch.tensor([-0.5, -0.5, 0.5, 0.5], dtype=torch.float64)
    own = torch.arange(vocab)[None] == t[4:, None]
    want = up[:, None] * (own * 1.0 - p)
    # p is off by (110 + 3 mean |d|) u of itself and more by 8 |d| u, |d| < 20 here
    tol = 0.5 * p * 400 * 2.0 ** -24 + (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * want.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert bool(((r.grad[4:].double().cpu() - want).abs() <= tol).all())


def test_a_gap_that_is_no_number():
    """Both impossible: no order between them, and the result says so."""
    x = torch.full((4,), -INF).cuda().requires_grad_()
    for smoothing in (0.0, 0.5, 1.0):
        r = L.preference_loss(x, torch.tensor([0, 2, 4]).cuda(), smoothing=smoothing)
        assert bool(r.loss.isnan().all()) and r.reward.tolist() == [[-INF, -INF]]
        assert bool(torch.autograd.grad(r.loss.sum(), x)[0].isnan().all())
