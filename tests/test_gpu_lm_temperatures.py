"""Temperatures from the least to the largest that the calls take, with gradients of both the log probability
and the entropy: 1 / T = 2^126 times a bounded number overflows only where the gradient itself does."""
import math

import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import losses as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(3, 1000), (3, 150001), (5, 16000), (260, 70000)])
@pytest.mark.parametrize("temperature", [2.0 ** -126, 2.0 ** -120, 1e-30, 1e-3, 1e3, 1e30, 2.0 ** 126])
def test_gradients_at_any_temperature(rows, vocab, dtype, temperature):
    g = torch.Generator().manual_seed(rows + vocab)
    x = torch.randn(rows, vocab, generator=g).mul(4).round().div(4)      # many ties at the top
    x[0] = -3.25                                           # one value: p = 1 / vocab at any temperature
    x = x.to(dtype).cuda()
    t = torch.randint(0, vocab, (rows,), generator=g)
    t[1] = -100
    t = t.cuda()
    gl, gh = torch.rand(rows, generator=g).cuda() * 0.5, torch.rand(rows, generator=g).cuda() * 0.5
    ref, tol = P.logprob_grad(x, t, gl, gh, temperature)
    # entries of p = 0 have gradient 0; elsewhere |gradient| T <= gl + gh (H + ln vocab) could pass the
    # type's largest value: those are compared below it only
    most = torch.finfo(dtype).max
    inside = ref.abs() < most / 2
    tol = torch.where(torch.isfinite(tol), tol, math.inf)
    half = P.half_step(dtype)
    lim = tol * (1 + half) + half * ref.abs() + P.smallest(dtype) + P.TINY
    one = L.token_logprobs_grad(x, t, gl, gh, temperature=temperature).grad
    xg = x.clone().requires_grad_()
    r = L.token_logprobs(xg, t, temperature=temperature)
    auto, = torch.autograd.grad((r.logprob, r.entropy), xg, (gl, gh))
    for grad in (one, auto):
        off = (grad.double() - ref).abs()
        assert not bool(torch.isnan(grad).any())
        assert bool((off <= lim)[inside].all()), (off / lim)[inside].max().item()
